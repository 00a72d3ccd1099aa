// paged_attention.cu -- attention over the e4m3 paged cache on the tcgen05 tensor cores: every token
// of a causal window, or the picked regions plus the row's own.
//
//   s_t = softmax_scale (q . kcode_t) kscale(region of t),  p = softmax(s),  out = sum_t p_t vscale vcode_t
//
// The codes go to the tensor cores as they lie in the cache (kind::f8f6f4), so nothing is converted
// on the way and a key costs half the bytes of bf16.  The other operand of each product is then e4m3
// too, which has 4 significant bits; q and p are therefore split into parts, each the e4m3 rounding
// of what the parts before it left, times 2^5: two parts hold a bf16 q (8 bits) exactly down to 2^-22
// of the head's largest value, three hold the 11 bits of a weight in f16, down to 2^-24 of the
// largest.  The parts are more columns of the small side of the product, which costs nothing at few
// heads: 128 keys are the M side,
//
//   S^T [128 keys x 2 H]  = K_tile [128 x 128 dims]       . (q parts)^T     (two TMEM buffers)
//   O^T [128 dims x 3 H] += V_tile^T [128 dims x 128 keys] . (p parts)^T
//
// with H query heads of one row.  A region (8 tokens x 128 B) is one 128-byte-swizzle atom: K-major A
// for the first product, MN-major A for the second, from one TMA box (pages whose length allows it
// come in boxes of up to 16 regions).
//
// Scales.  kscale multiplies the fp32 score.  vscale joins the weight before it is split, relative to
// a power of two not below any vscale so far, so that the parts' range is spent on what a key adds to
// the output; the row sum takes the weight without it.
//
// Work.  An item is a (row, group).  Few items are cut into equal parts, many have their tiles laid
// end to end and cut into equal runs, so that a ragged batch, one long row and a chunk of many rows
// all fill the GPU; a second kernel joins the items that CTAs share, in CTA order (the bits do not
// depend on timing).
//
// A CTA: four softmax warps (a key to a thread), a warp for each product (so that neither waits for
// what the other waits for), two warps that look the regions up (page, scales) a few tiles ahead and
// issue the copies, K a tile ahead of V, and leave what the softmax needs of each region in a small
// ring.
//
// What bounds it, with 4 KV groups of 8 heads and pages of 64 tokens, join included:
//   one row of 1M tokens        160 us  1.08 GB, 6.73 TB/s: the copy bandwidth of HBM
//   16 rows of 16K to 32K        68 us  404 MB, 6.0 TB/s: HBM, and the last CTA's tail
//   one row of 4,608 tokens     9.3 us  latency: split 2, page, scale and key loads 2, one tile 1,
//                                       second product and states 1.3, launch and join 3
//   16 rows of 512 picks       23.7 us  the copies alone 22.3 (68 MB in boxes of 1 KB)
//   2,048 rows of 512 picks   1,135 us  the copies alone 934: 8.6 GB in boxes of 1 KB out of L2,
//                                       one in 32 cycles on each SM
#include "paged_device.cuh"

namespace step5 {

namespace {

constexpr int kTile = 16;            // regions of a tile
constexpr int kSoft = 128;           // softmax threads
constexpr int kThreads = kSoft + 64 + 64;
constexpr int kQkWarp = 4, kLoadWarp = 6, kLoadWarps = 2;  // (the second product's warp is 5)
constexpr int kRing = 8;             // tiles whose scales and masks are in shared memory
constexpr uint32_t kSlotBytes = kTile * 1024;
constexpr float kSlack = 3.0f;       // log2 units a tile's maximum may pass the running one by
constexpr float kPTop = 32.0f;       // weights are split from p * 2^(8 - slack): at most 2^8, whose parts fit e4m3

// MANY: for launches of many items, three CTAs an SM with few slots, which hide one another's latency
// (2,048 rows of 512 picks: 1,130 us against 1,380 with two, 256 rows 157 against 185); for few items
// two CTAs with more copies in flight and fewer states to join (one row of 512 picks: 9.5 us against
// 10.2 with three; 16 rows 23.7 against 23.4).
template <int H_, bool PICKS_, bool MANY_>
struct Shape {
    static constexpr int H = H_;                       // query heads of a group
    static constexpr bool PICKS = PICKS_;
    static constexpr int NS = 2 * H < 16 ? 16 : 2 * H;
    static constexpr int NO = (3 * H + 15) / 16 * 16;
    static constexpr int kCtas = MANY_ && H <= 8 ? 3 : 2;  // per SM
    static constexpr int kSlots = kCtas == 3 ? 3 : 5;
    static_assert(kSlots <= 6, "the barriers of copies and the ring are reused after 4 and 8 tiles");
    static constexpr uint32_t kCols = 2 * NS + NO <= 64 ? 64 : 128;
    static constexpr uint32_t kQBytes = NS * 128, kPBytes = 128 * NO;
    static constexpr uint32_t kPGroup = 8 * NO;        // bytes of 8 keys of P
    static constexpr uint32_t kSmem = 1024 + kSlots * kSlotBytes + kQBytes + 2 * kPBytes;
    static constexpr uint32_t kIdesc1 = tc::instr_desc(tc::kFmtE4M3, false, false, 128, NS);
    static constexpr uint32_t kIdesc2 = tc::instr_desc(tc::kFmtE4M3, true, true, 128, NO);
    static constexpr int kState = H * 130;             // floats of a partial state: m[H], l[H], o[H][128]
};

// Reduction of NV values per lane (a power of two <= 32) over the warp, one shuffle per halving:
// lane pairs split the values between them.  *idx: which value this lane ends up with.
template <int NV, int M, class Op>
__device__ __forceinline__ float fold(float* w, int lane, int* idx, Op op) {
    if constexpr (M == 0) {
        return w[0];
    } else if constexpr (NV > 1) {
        const bool up = (lane & M) != 0;
#pragma unroll
        for (int j = 0; j < NV / 2; ++j) {
            const float send = up ? w[j] : w[j + NV / 2];
            const float keep = up ? w[j + NV / 2] : w[j];
            w[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, M));
        }
        if (up) *idx += NV / 2;
        return fold<NV / 2, M / 2>(w, lane, idx, op);
    } else {
        w[0] = op(w[0], __shfl_xor_sync(0xffffffffu, w[0], M));
        return fold<1, M / 2>(w, lane, idx, op);
    }
}
struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// An item: the keys of row n in group g, tiles of 16 entries.  Without picks entry e is region
// r0 + e (r0 a multiple of the box), with picks the e-th pick and the own region behind them.
struct Item {
    int n, g;
    int b;               // sequence; -1: padding (no tiles), -2: out of range (one empty tile, its output zero)
    int lo, hi;          // first and last token
    int r0, entries, tiles;
};

template <bool PICKS>
__device__ __forceinline__ Item item_at(const PagedAttnParams& p, int i) {
    Item it;
    it.g = i / p.N;
    it.n = i - it.g * p.N;
    it.b = p.row_seq[it.n];
    it.hi = p.row_pos[it.n];
    it.lo = it.r0 = it.entries = it.tiles = 0;
    if (it.b == -1) return it;
    if (it.b < 0 || it.b >= p.B || it.hi < 0 || it.hi >= p.pages.page_tokens * p.pages.table_len) {  // (fits int32)
        it.b = -2;
        it.tiles = 1;
        return it;
    }
    if (PICKS) {
        it.entries = min(max(p.sel_count[(int64_t)it.n * p.G + it.g], 0), p.top_k) + 1;
    } else {
        it.lo = p.window > 0 ? max(0, it.hi - p.window + 1) : 0;
        it.r0 = (it.lo >> 3) & ~(p.box_regions - 1);
        it.entries = (it.hi >> 3) - it.r0 + 1;
    }
    it.tiles = (it.entries + kTile - 1) / kTile;
    return it;
}

// What the softmax needs of a region of the tile.
struct __align__(16) Meta {
    float ks, vs;
    uint32_t mask;    // its tokens that the row sees
    uint32_t loaded;  // 1: a copy brings its codes
};

// The output v of a (row, head), number `at` of them, through its gate.
__device__ __forceinline__ float gated(const PagedAttnParams& p, int64_t at, float v) {
    return v * (1.0f / (1.0f + expf(-bf16_to_f32(p.gate[at]))));
}

template <class S>
__global__ void __launch_bounds__(kThreads, S::kCtas)
    paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      PagedAttnParams p) {
    constexpr int H = S::H;
    constexpr bool PICKS = S::PICKS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw, 1024);
    uint8_t* slots = smem;
    uint8_t* qt = smem + S::kSlots * kSlotBytes;
    uint8_t* pt = qt + S::kQBytes;
    __shared__ __align__(8) uint64_t kfull[4], vfull[4], empty[S::kSlots], sbar[2], obar[2], pbar[2], qbar;
    __shared__ Meta ring[kRing][kTile];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    __shared__ int s_note[kRing];  // of a tile: MMA steps | first tile of a segment << 8
    __shared__ float red[3][4][H + 1];
    __shared__ __align__(16) float s_cq[2][H];
    __shared__ int64_t s_scan[kThreads / 32];
    __shared__ int s_tiles[kThreads], s_item, s_off, s_run, s_first, s_last;
    __shared__ Item s_it;  // item s_item
    __shared__ uint32_t s_ctas[kThreads / 32][32];

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int items = p.N * p.G;

    if (tid == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        // a slot's two readers are different warps, so a copy's arrival is told by tile, not by slot:
        // a warp that waited by slot would miss every other phase of it (tile t + 4 is not copied
        // before tile t is used)
        for (int s = 0; s < 4; ++s) {
            mbar_init(&kfull[s], kLoadWarps);
            mbar_init(&vfull[s], kLoadWarps);
        }
        for (int s = 0; s < S::kSlots; ++s) mbar_init(&empty[s], 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sbar[s], 2);
            mbar_init(&obar[s], 1);
            mbar_init(&pbar[s], kSoft / 32);
        }
        mbar_init(&qbar, kSoft / 32);
        fence_mbar_init();
        s_fail = 0;
    }
    if (warp == 0) tc::alloc(&s_tmem, S::kCols);
    if (2 * H < S::NS)  // q rows that no head fills (softmax threads, which fence them below)
        for (int i = tid; i < (int)(S::NS - 2 * H) * 8; i += kSoft)
            if (tid < kSoft) reinterpret_cast<uint4*>(qt + 2 * H * 128)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_launch_dependents();

    // This CTA's run of tiles, from tile off0 of item item0 on.
    int64_t start = 0, per = 1;  // (many items: the run's first tile among all, tiles of a run)
    const bool few = 2 * items <= (int)gridDim.x;
    if (few) {
        // Few items: each is cut into equal parts, one CTA a part, of at most L tiles for the
        // smallest L of 32 tried that needs no more CTAs than there are (2 L0 always does).  No CTA
        // then has parts of two items. (fewer than 2^8 items of at most 2^24 tiles)
        Item own{};
        if (tid < items) own = item_at<PICKS>(p, tid);
        const uint32_t mine = (uint32_t)own.tiles;
        s_tiles[tid] = own.tiles;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) s_scan[warp] = sum;
        if (tid == 0) s_run = 0;
        __syncthreads();
        uint32_t total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) total += (uint32_t)s_scan[w];
        const uint32_t least = max(1u, total / gridDim.x + (total % gridDim.x ? 1u : 0u));
        uint32_t most = least + (least * (uint32_t)lane + 30u) / 31u;  // this lane's L
        uint32_t ctas = 0;
        for (int i = warp; i < items; i += kThreads / 32) ctas += ((uint32_t)s_tiles[i] + most - 1u) / most;
        s_ctas[warp][lane] = ctas;
        __syncthreads();
        ctas = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) ctas += s_ctas[w][lane];
        most = __shfl_sync(0xffffffffu, most, __ffs(__ballot_sync(0xffffffffu, ctas <= gridDim.x)) - 1);
        const int parts = (int)((mine + most - 1u) / most);
        int inc = parts;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int first = inc - parts;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w)
            if (w < warp) first += (int)s_scan[w];
        const int part = (int)blockIdx.x - first;
        if (part >= 0 && part < parts) {
            s_item = tid;
            s_it = own;
            const uint32_t each = mine / (uint32_t)parts, more = mine % (uint32_t)parts;  // (the first ones take one more)
            s_off = (int)((uint32_t)part * each + min((uint32_t)part, more));
            s_run = (int)(each + ((uint32_t)part < more ? 1u : 0u));
            s_first = first;
            s_last = first + parts - 1;
            if (part == 0) p.shared_items[tid] = make_int4(0, 0, 0, -1);  // (again below if it has several parts)
        }
        if (blockIdx.x == 0 && tid < items && mine == 0) p.shared_items[tid] = make_int4(0, 0, 0, -1);
    } else {
        // Many: the items' tiles are laid end to end and every CTA takes an equal run of them.
        if (tid == 0) {
            p.shared_items[blockIdx.x] = make_int4(0, 0, 0, -1);  // (again below if an item that other CTAs share begins here)
            s_run = 0;
        }
        const int chunk = (items + kThreads - 1) / kThreads;
        const int i0 = min(items, tid * chunk), i1 = min(items, i0 + chunk);
        int64_t sum = 0;
        for (int i = i0; i < i1; ++i) sum += item_at<PICKS>(p, i).tiles;
        int64_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int64_t before = inc - sum, total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        per = (total + gridDim.x - 1) / gridDim.x;
        start = blockIdx.x * per;
        if (start >= before && start < before + sum) {
            int64_t at = before;
            for (int i = i0; i < i1; ++i) {
                const Item it = item_at<PICKS>(p, i);
                const int t = it.tiles;
                if (start < at + t) {
                    s_item = i;
                    s_it = it;
                    s_off = (int)(start - at);
                    s_run = (int)min(per, total - start);
                    break;
                }
                at += t;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const int run = s_run, item0 = s_item, off0 = s_off;

    if (run == 0) {
        // nothing to do
    } else if (warp >= kLoadWarp) {
        // ---------------- load warps: K_0, K_1, V_0, K_2, V_1, ... over the run's tiles, each into
        // the next slot once the product that read it is done.  Warp lw takes entries 8 lw .. 8 lw +
        // 7 of a tile.
        const int lw = warp - kLoadWarp;
        const int k = p.box_regions;  // (a box of 16 regions is the first warp's)
        const int q = lw * 8 + (lane & 7);                // this lane's entry
        const bool boxes = lane < 8 && (q & (k - 1)) == 0;
        bool ok = true;
        int j = 0;  // slot uses so far
        Item it{};
        int nitem = item0, at = 0;       // next item, this one's tile
        int left = run, in_seg = 0;      // tiles of the run, of the segment, not yet walked
        // Lane l looks up its entry in tile l / 8 of four tiles, in three steps (region; pool row;
        // scales), the next four while these go by.
        int b_r = 0, b_row = -1, n_r = 0, n_row = -1, batch = -1, done = 0;
        float b_ks = 0.0f, b_vs = 0.0f, n_ks = 0.0f, n_vs = 0.0f;
        bool fresh = false;  // n_ks, n_vs are the batch's
        const int32_t* ids = nullptr;
        auto look = [&](int of, int steps) {
            const int e = (of * 4 + (lane >> 3)) * kTile + q;
            if (steps & 1) {
                n_r = -1;
                if (PICKS) {
                    if (e < it.entries) n_r = e == it.entries - 1 ? it.hi >> 3 : ids[e];
                } else if (it.b >= 0 && e < (it.entries + k - 1) / k * k && ((it.r0 + e) | (k - 1)) >= (it.lo >> 3)) {
                    n_r = it.r0 + e;  // (with its box, of which some region is the row's)
                }
            }
            if (steps & 2) {
                n_row = -1;
                bool bad = false;
                if (PICKS) bad = e < it.entries && (n_r < 0 || n_r > it.hi >> 3 || (n_r == it.hi >> 3) != (e == it.entries - 1));
                if (!bad && n_r >= 0) {
                    n_row = (int)page_row(p.pages, p.G, it.b, it.g, n_r * 8);
                    bad = n_row < 0;
                }
                if (bad) raise_status(p.status, kDevRange);
            }
            if (steps & 4) {
                n_ks = n_vs = 0.0f;
                if (n_row >= 0) {
                    n_ks = p.k_scales[n_row >> 3];
                    n_vs = p.v_scales[n_row >> 3];
                }
            }
        };
        // Tile t's K (and its ring entry) or V.
        auto put = [&](bool isv, int row, int note, uint32_t zero, int t) {
            const int slot = j % S::kSlots, use = j / S::kSlots;
            if (use > 0 && !wait(&empty[slot], (uint32_t)((use - 1) & 1))) ok = false;
            if (*reinterpret_cast<volatile int*>(&s_fail) != 0) ok = false;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                return;
            }
            ++j;
            uint8_t* dst = slots + slot * kSlotBytes;
            if (isv && zero != 0) {  // regions of V inside the product's steps that no copy fills
                for (uint32_t z = zero; z; z &= z - 1) {
                    uint4* to = reinterpret_cast<uint4*>(dst + (__ffs(z) - 1) * 1024);
                    to[lane] = make_uint4(0, 0, 0, 0);
                    to[lane + 32] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
            }
            uint64_t* full = isv ? &vfull[t & 3] : &kfull[t & 3];
            const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) expect_tx(full, (uint32_t)__popc(have) * 1024u * k);
            __syncwarp();
            if (row >= 0) tma_load_2d(dst + q * 1024, isv ? &vmap : &kmap, full, 0, row);
            if (!isv) {
                // (this slot was free, so the softmax is past tile t - 5 and the ring's entry is free
                // too; the copies are on their way while the scales of a segment's first tile come)
                if (fresh) b_ks = n_ks, b_vs = n_vs, fresh = false;
                if (lane >> 3 == (at & 3)) {
                    const int t0 = b_r * 8;
                    const int a = min(max(it.lo - t0, 0), 8), z = min(max(it.hi - t0 + 1, 0), 8);
                    uint32_t mask = b_row >= 0 && z > a ? ((1u << z) - 1u) & ~((1u << a) - 1u) : 0u;
                    if (mask && !(scale_ok(b_ks) && scale_ok(b_vs))) {
                        raise_status(p.status, kDevRange);
                        mask = 0;
                    }
                    ring[t & (kRing - 1)][q] = Meta{b_ks, b_vs, mask, b_row >= 0 ? 1u : 0u};
                }
                if (lw == 0 && lane == 0) s_note[t & (kRing - 1)] = note;
                __syncwarp();
            }
            if (lane == 0) arrive(full);
        };
        int row = -1;  // of the tile whose V is next
        uint32_t zero = 0;
        int off = off0;
        for (int t = 0; t <= run && ok; ++t) {
            int nrow = -1, nnote = 0;
            uint32_t nzero = 0;
            if (t < run) {
                const bool first = in_seg == 0;
                if (first) {  // the next segment
                    it = s_it;
                    if (t > 0) {
                        it.tiles = 0;
                        while (nitem < items && (it = item_at<PICKS>(p, nitem)).tiles <= off) ++nitem;
                    }
                    if (nitem >= items) {  // (the rows have changed under the kernel)
                        ok = false;
                        break;
                    }
                    ++nitem;
                    if (PICKS) ids = p.sel_ids + ((int64_t)it.n * p.G + it.g) * p.top_k;
                    at = off;
                    in_seg = min(it.tiles - off, left);
                    left -= in_seg;
                    off = 0;
                    batch = -1, done = 0;
                } else {
                    ++at;
                }
                --in_seg;
                if (batch != at >> 2) {
                    if (done != 7) look(at >> 2, 7 & ~done);
                    batch = at >> 2;
                    b_r = n_r, b_row = n_row, fresh = true, done = 0;
                } else if ((batch + 1) * 4 < it.tiles) {
                    const int todo = ((2 << (at & 3)) / 2 - 1) & ~done;  // one more step at tiles 1, 2 and 3
                    look(batch + 1, todo);
                    done |= todo;
                }
                nrow = __shfl_sync(0xffffffffu, b_row, (at & 3) * 8 + (lane & 7));
                const uint32_t got = __ballot_sync(0xffffffffu, lane < 8 && nrow >= 0) & 0xffu;
                if (!boxes) nrow = -1;
                const int steps = it.b < 0 ? 0 : min(4, (it.entries - at * kTile + 3) >> 2);
                // a box of several regions is copied whole or not at all; every entry of it has its row
                nzero = (~got << (lw * 8)) & (0xffu << (lw * 8)) & ((1u << (4 * steps)) - 1u);
                nnote = steps | (first ? 256 : 0);
                put(false, nrow, nnote, 0, t);
            }
            if (t > 0 && ok) put(true, row, 0, zero, t - 1);
            row = nrow, zero = nzero;
        }
        if (!ok) {
            // a wait gave up: let the copies issued land (bounded) before the shared memory goes away
            if (lane == 0) {
                raise_status(p.status, kDevTimeout);
                atomicExch(&s_fail, 1);
                const int nk = min(run, (j + 2) / 2), nv = j - nk;  // K and V copies issued
                for (int i = max(0, nk - 4); i < nk; ++i) wait(&kfull[i & 3], (uint32_t)((i >> 2) & 1));
                for (int i = max(0, nv - 4); i < nv; ++i) wait(&vfull[i & 3], (uint32_t)((i >> 2) & 1));
            }
            __syncwarp();
        }
    } else if (warp >= kQkWarp) {
        // ---------------- product warps: K_t is slot use 2 t - 1 (0 for t = 0), V_t use 2 t + 2 (one
        // less for the last tile, which no K follows)
        const bool qk = warp == kQkWarp;
        const uint32_t slot_addr = smem_u32(slots), p_addr = smem_u32(pt);
        const uint64_t dq = tc::smem_desc(smem_u32(qt), 16, 1024, tc::kSwizzle128);
        bool ok = true;
        uint64_t* last_commit = nullptr;
        uint32_t last_parity = 0;
        int seg = 0;
        for (int t = 0; t < run; ++t) {
            const int j = qk ? (t == 0 ? 0 : 2 * t - 1) : (t + 1 < run ? 2 * t + 2 : 2 * t + 1), slot = j % S::kSlots;
            if (!wait(qk ? &kfull[t & 3] : &vfull[t & 3], (uint32_t)((t >> 2) & 1))) ok = false;
            const int note = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_note[t & (kRing - 1)]), 0);
            // First product: tile t - 2 is through (its S has been read, and its P, which the softmax
            // of tile t overwrites); q of a segment's first tile is there.  Second: P_t is there.
            if (qk) {
                if (t >= 2 && !wait(&obar[t & 1], (uint32_t)(((t - 2) >> 1) & 1))) ok = false;
                if ((note & 256) && !wait(&qbar, (uint32_t)(seg++ & 1))) ok = false;
            } else {
                if (!wait(&pbar[t & 1], (uint32_t)((t >> 1) & 1))) ok = false;
            }
            if (*reinterpret_cast<volatile int*>(&s_fail) != 0) ok = false;
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc::fence_after_sync();
            const uint64_t da = tc::smem_desc(slot_addr + slot * kSlotBytes, 16, 1024, tc::kSwizzle128);
            if (qk) {
                if (elect()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 32 dims each
                        tc::mma_f8(tmem + (uint32_t)(S::NS * (t & 1)), da + 2 * i, dq + 2 * i, S::kIdesc1, i > 0);
                    arrive(&sbar[t & 1]);  // (hands the tile's ring entry on, which came with its K)
                    tc::commit(&sbar[t & 1]);
                    tc::commit(&empty[slot]);
                }
            } else {
                const uint64_t db = tc::smem_desc(p_addr + (uint32_t)(t & 1) * S::kPBytes, S::kPGroup, 128, tc::kSwizzleNone);
                if (elect()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 32 keys (four regions) each
                        if (i < (note & 255))
                            tc::mma_f8(tmem + 2u * S::NS, da + 256u * i, db + (uint32_t)(S::kPGroup >> 2) * i, S::kIdesc2,
                                       !(note & 256) || i > 0);
                    tc::commit(&obar[t & 1]);
                    tc::commit(&empty[slot]);
                }
            }
            __syncwarp();
            last_commit = &empty[slot];
            last_parity = (uint32_t)((j / S::kSlots) & 1);
        }
        if (!ok) {
            if (lane == 0) {
                raise_status(p.status, kDevTimeout);
                atomicExch(&s_fail, 1);
                if (last_commit) wait(last_commit, last_parity);
            }
            __syncwarp();
        }
    } else {
        // ---------------- softmax warps: one key per thread (its TMEM lane)
        const int key = tid, q = key >> 3;
        const uint32_t lanes = tc::taddr(tmem, warp * 32, 0);
        float2 neg_m[H / 2], l_part[H / 2];  // less the running maxima, the row sums of this thread's keys
        float vref = 0.0f, vinv = 0.0f;
        Item it{}, done{};  // the segment's item; that of the segment before, for its epilogue
        int64_t done_begin = 0;
        bool whole = true, begins = true;  // it has the whole item, its first tile
        bool failed = false;
        int t = 0;  // tile of the run

        auto give_up = [&] {
            raise_status(p.status, kDevTimeout);
            atomicExch(&s_fail, 1);
        };

        // The item's heads as two e4m3 parts each: 16 lanes to a head.
        auto build_q = [&](float* cq) {
#pragma unroll
            for (int u0 = 0; u0 < H; u0 += 8) {
                const int u = u0 + (tid >> 4), d8 = tid & 15;
                if (H < 8 && u >= H) break;  // (whole warps)
                uint4 x = make_uint4(0, 0, 0, 0);
                if (it.b >= 0)
                    x = *reinterpret_cast<const uint4*>(p.q + ((int64_t)it.n * p.Hq + (int64_t)it.g * H + u) * 128 + d8 * 8);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t a = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) a = max(a, max(xs[i] & 0x7fffu, (xs[i] >> 16) & 0x7fffu));
#pragma unroll
                for (int d = 8; d; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
                const bool finite = a < 0x7f80u;
                // q * 2^(7 - e) is below 2^8 for the largest |q|, whose exponent is e
                const int e = a == 0 ? 0 : max((int)(a >> 7) - 127, -100);
                const float up = __uint_as_float((uint32_t)(min(7 - e, 120) + 127) << 23);
                if (d8 == 0) cq[u] = finite ? p.scale_log2 / up : __int_as_float(0x7fc00000);
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // (f16 holds a bf16 below 2^8 exactly down to 2^-17, 2^-24 of the head's largest)
                    __half2 x2 = __floats2half2_rn(bf16_lo(xs[i]) * up, bf16_hi(xs[i]) * up);
                    hi[i >> 1] |= next_part(x2) << (16 * (i & 1));
                    lo[i >> 1] |= last_part(x2) << (16 * (i & 1));
                }
                auto to = [&](int r) {
                    return reinterpret_cast<uint2*>(qt + r * 128 + (((d8 >> 1) ^ (r & 7)) << 4) + (d8 & 1) * 8);
                };
                *to(u) = make_uint2(hi[0], hi[1]);
                *to(H + u) = make_uint2(lo[0], lo[1]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(&qbar);
        };

        // O of the segment that ended with tile t - 1, and its output or partial state.
        auto epilogue = [&] {
            const int tl = t - 1;
            float(&rd)[4][H + 1] = red[2];
            int hidx = 0;
            float l[H];
#pragma unroll
            for (int h = 0; h < H; ++h) l[h] = h & 1 ? l_part[h / 2].y : l_part[h / 2].x;
            const float sum = fold<H, 16>(l, lane, &hidx, Add{});
            if ((lane & (32 / H - 1)) == 0) rd[warp][hidx] = sum;
            const bool w_ok = wait(&obar[tl & 1], (uint32_t)((tl >> 1) & 1));
            tc::fence_after_sync();
            if (!w_ok) give_up();
            if (group_or(1, kSoft, !w_ok || *reinterpret_cast<volatile int*>(&s_fail) != 0)) {
                failed = true;
                return;
            }
            float o[H], a[16], b[16];
            const uint32_t ob = lanes + 2 * S::NS;
            tc::ld16(ob, a);
            if constexpr (H >= 8) tc::ld16(ob + 16, b);
            if constexpr (H == 16) {
                float c[16];
                tc::ld16(ob + 32, c);
#pragma unroll
                for (int h = 0; h < H; ++h) o[h] = a[h] + (b[h] + c[h] * (1.0f / kPart)) * (1.0f / kPart);
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h)
                    o[h] = a[h] + (a[H + h] + (H == 8 ? b[h] : a[(2 * H + h) & 15]) * (1.0f / kPart)) * (1.0f / kPart);
            }
            float L[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                L[h] = (rd[0][h] + rd[1][h]) + (rd[2][h] + rd[3][h]);
                // (vref apart: the quotient may underflow with it)
                o[h] = L[h] == 0.0f ? 0.0f : o[h] * __fdividef(1.0f / kPTop, L[h]) * vref;
            }
            if (whole) {
                const int64_t at = (int64_t)done.n * p.Hq + (int64_t)done.g * H;
                if (p.gate != nullptr && L[0] != 0.0f)  // (without keys no head has a weight, and zero stays zero)
#pragma unroll
                    for (int h = 0; h < H; ++h) o[h] = gated(p, at + h, o[h]);
#pragma unroll
                for (int h = 0; h < H; ++h) p.out[(at + h) * 128 + key] = f32_to_bf16_bits(o[h]);
            } else {  // CTAs first .. last share the item; each leaves its state, which the join kernel reads
                float* st = p.states + ((int64_t)2 * blockIdx.x + (begins ? 1 : 0)) * S::kState;
#pragma unroll
                for (int h = 0; h < H; ++h) st[2 * H + h * 128 + key] = o[h];
                if (key == 0)
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        st[h] = -(h & 1 ? neg_m[h / 2].y : neg_m[h / 2].x);
                        st[H + h] = L[h];
                    }
            }
            if (!whole && begins && tid == 0) {
                if (few)
                    p.shared_items[item0] = make_int4(done.n, done.g, s_first, s_last);
                else
                    p.shared_items[blockIdx.x] = make_int4(done.n, done.g, (int)blockIdx.x, (int)((done_begin + done.tiles - 1) / per));
            }
        };

        int segs = 0, nitem = item0, off = off0;
        for (int left = run; left > 0;) {
            it = s_it;
            if (t > 0) {
                it.tiles = 0;
                while (nitem < items && (it = item_at<PICKS>(p, nitem)).tiles <= off) ++nitem;
            }
            if (nitem >= items) {
                give_up();
                failed = true;
                break;
            }
            ++nitem;
            float* cq = s_cq[segs++ & 1];
            build_q(cq);
            if (t > 0)
                epilogue();
            else
                group_or(1, kSoft, false);  // (cq is written)
            if (failed) break;
            if (tid == 0) {
                if (it.b == -2) raise_status(p.status, kDevRange);
                if (PICKS && it.b >= 0) {
                    const int n = p.sel_count[(int64_t)it.n * p.G + it.g];
                    if (n < 0 || n > p.top_k) raise_status(p.status, kDevRange);
                }
            }
            const int seg = min(it.tiles - off, left);
            done = it;
            done_begin = start + (run - left) - off;
            whole = seg == it.tiles;
            begins = off == 0;
            left -= seg;
            off = 0;
            vref = vinv = 0.0f;
#pragma unroll
            for (int h = 0; h < H / 2; ++h) {
                neg_m[h] = both(INFINITY);
                l_part[h] = both(0.0f);
            }
            for (int i = 0; i < seg; ++i, ++t) {
                // (tile t - 2's second product is done too: the first product of this one waited for it)
                bool w_ok = wait(&sbar[t & 1], (uint32_t)((t >> 1) & 1));
                tc::fence_after_sync();
                const Meta me = ring[t & (kRing - 1)][q];
                const bool sees = (me.mask >> (key & 7) & 1u) != 0;
                // s[h] = q . kcode kscale; its logit in log2 units is s[h] cq[h], y[h] that less the
                // running maximum
                float2 s[H / 2], y[H / 2];
                const uint32_t sb = lanes + (uint32_t)(S::NS * (t & 1));
                {
                    float x[16], z[16];
                    tc::ld16(sb, x);
                    if constexpr (H == 16) tc::ld16(sb + H, z);
#pragma unroll
                    for (int h = 0; h < H; h += 2) {
                        const float2 lo = H == 16 ? make_float2(z[h], z[h + 1]) : make_float2(x[(H + h) & 15], x[(H + h + 1) & 15]);
                        s[h / 2] = mul2(fma2(lo, both(1.0f / kPart), make_float2(x[h], x[h + 1])), both(me.ks));
                    }
                }
                float top = -INFINITY;
#pragma unroll
                for (int h = 0; h < H; h += 2) {
                    y[h / 2] = fma2(s[h / 2], *reinterpret_cast<const float2*>(cq + h), neg_m[h / 2]);
                    top = fmaxf(top, fmaxf(y[h / 2].x, y[h / 2].y));
                }
                // The running maxima move when a key passes one by more than the slack, vref when a
                // vscale passes it; l and O are rescaled then.  Every softmax thread takes the same
                // steps.
                if (!w_ok) give_up();
                if (__builtin_expect(group_or(1, kSoft, (sees && (top > kSlack || me.vs > vref)) || !w_ok), 0)) {
                    if (*reinterpret_cast<volatile int*>(&s_fail) != 0) failed = true;
                    float alpha[H];
                    int hidx = 0;
#pragma unroll
                    for (int h = 0; h < H; ++h) alpha[h] = sees ? (h & 1 ? s[h / 2].y : s[h / 2].x) * cq[h] : -INFINITY;
                    const float wmax = fold<H, 16>(alpha, lane, &hidx, Max{});
                    const uint32_t vmax = __reduce_max_sync(0xffffffffu, sees ? __float_as_uint(me.vs) : 0u);
                    float(&rd)[4][H + 1] = red[t & 1];
                    if ((lane & (32 / H - 1)) == 0) rd[warp][hidx] = wmax;
                    if (lane == 0) rd[warp][H] = __uint_as_float(vmax);
                    if (group_or(1, kSoft, failed)) {
                        failed = true;
                        break;
                    }
                    float ratio = 1.0f;
                    const float old = vref, v = fmaxf(fmaxf(rd[0][H], rd[1][H]), fmaxf(rd[2][H], rd[3][H]));
                    if (v > vref) {
                        const uint32_t u = __float_as_uint(v);
                        const float next = __uint_as_float((u & 0x7f800000u) + ((u & 0x7fffffu) ? 0x800000u : 0u));
                        vref = next;
                        vinv = __uint_as_float(0x7f000000u - __float_as_uint(next));  // (exact: next is 2^-126 .. 2^126)
                        ratio = old * vinv;
                    }
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float tmax = fmaxf(fmaxf(rd[0][h], rd[1][h]), fmaxf(rd[2][h], rd[3][h]));
                        float& neg = h & 1 ? neg_m[h / 2].y : neg_m[h / 2].x;
                        float& l = h & 1 ? l_part[h / 2].y : l_part[h / 2].x;
                        const bool moves = tmax > kSlack - neg || (neg == INFINITY && tmax > -INFINITY);
                        const float a = ex2(-neg - tmax);
                        alpha[h] = moves ? a : 1.0f;
                        neg = moves ? -tmax : neg;
                        l *= alpha[h];
                    }
#pragma unroll
                    for (int h = 0; h < H; h += 2)
                        y[h / 2] = fma2(s[h / 2], *reinterpret_cast<const float2*>(cq + h), neg_m[h / 2]);
                    if (i > 0) {
                        w_ok = wait(&obar[(t - 1) & 1], (uint32_t)(((t - 1) >> 1) & 1));
                        tc::fence_after_sync();
#pragma unroll
                        for (int c = 0; c < S::NO; c += 16) {
                            float o[16];
                            tc::ld16(lanes + 2 * S::NS + c, o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] *= alpha[x % H] * ratio;
                            tc::st16(lanes + 2 * S::NS + c, o);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, !sees)) {  // (a key that is not seen may have anything for a score)
#pragma unroll
                    for (int h = 0; h < H / 2; ++h) y[h] = sees ? y[h] : both(-INFINITY);
                }
                const float2 vf = both(sees ? me.vs * vinv * kPTop : 0.0f);
                uint32_t part[3][H / 4];
#pragma unroll
                for (int h = 0; h < H; h += 2) {
                    const float2 w = make_float2(ex2(y[h / 2].x), ex2(y[h / 2].y));
                    l_part[h / 2] = add2(l_part[h / 2], w);
                    // f16 keeps 11 bits of a weight (half a step is at most 2^-11 of it), the parts
                    // all of them
                    __half2 x = __float22half2_rn(mul2(w, vf));
                    const uint32_t a = next_part(x), b = next_part(x), c = last_part(x);
                    if (h % 4 == 0)
                        part[0][h / 4] = a, part[1][h / 4] = b, part[2][h / 4] = c;
                    else
                        part[0][h / 4] = __byte_perm(part[0][h / 4], a, 0x5410), part[1][h / 4] = __byte_perm(part[1][h / 4], b, 0x5410),
                        part[2][h / 4] = __byte_perm(part[2][h / 4], c, 0x5410);
                }
                uint8_t* pb = pt + (t & 1) * S::kPBytes + q * S::kPGroup + (key & 7) * 16;
                if constexpr (H == 16) {
#pragma unroll
                    for (int x = 0; x < 3; ++x)
                        *reinterpret_cast<uint4*>(pb + x * 128) = make_uint4(part[x][0], part[x][1], part[x][2], part[x][3]);
                } else if constexpr (H == 8) {
                    *reinterpret_cast<uint4*>(pb) = make_uint4(part[0][0], part[0][1], part[1][0], part[1][1]);
                    *reinterpret_cast<uint4*>(pb + 128) = make_uint4(part[2][0], part[2][1], 0u, 0u);
                } else {
                    *reinterpret_cast<uint4*>(pb) = make_uint4(part[0][0], part[1][0], part[2][0], 0u);
                }
                // a copied V row that the row does not see is zeroed: the cache may hold anything
                // there, and a zero weight must meet a finite value
                if (__builtin_expect(me.loaded && !sees, 0)) {
                    const int slot = (t + 1 < run ? 2 * t + 2 : 2 * t + 1) % S::kSlots;
                    w_ok &= wait(&vfull[t & 3], (uint32_t)((t >> 2) & 1));
                    uint4* vr = reinterpret_cast<uint4*>(slots + slot * kSlotBytes + key * 128);
#pragma unroll
                    for (int x = 0; x < 8; ++x) vr[x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                tc::fence_before_sync();
                if (!w_ok) give_up();  // (the warps leave together at the next barrier)
                __syncwarp();
                if (lane == 0) arrive(&pbar[t & 1]);
            }
            if (failed) break;
        }
        if (!failed) epilogue();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, S::kCols);
}

// Joins the items that CTAs of the launch before shared: a block per (entry of shared_items, head),
// its threads' groups of 128 dims taking every GROUPS-th state, eight of them asked for before the
// weights are known (the states lie in L2; the join is latency, not bandwidth).  The sums run in an
// order fixed by the CTAs.
// Eight groups for few blocks, two for many (one row of 4,608 tokens: 9.3 us in all against 11.4 with
// two; 16 rows of 512 picks: 23.7 against 28.8 with eight).
template <class S, int GROUPS>
__global__ void __launch_bounds__(128 * GROUPS) join_kernel(PagedAttnParams p) {
    __shared__ float sw[kPagedMaxCtas], sm[GROUPS * 4], so[GROUPS][128], sl[GROUPS];
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.y, tid = threadIdx.x, d = tid & 127, grp = tid >> 7;
    const int4 item = p.shared_items[blockIdx.x];
    const int first = item.z, n = item.w - first + 1;
    if (item.w < 0) return;
    auto state = [&](int i) { return p.states + ((int64_t)2 * (first + i) + (i == 0 ? 1 : 0)) * S::kState; };
    constexpr int kDeep = 8;
    float v[kDeep];
#pragma unroll
    for (int x = 0; x < kDeep; ++x) v[x] = grp + x * GROUPS < n ? state(grp + x * GROUPS)[2 * S::H + c * 128 + d] : 0.0f;
    // the states' weights 2^(m - M) l
    float M = -INFINITY;
    for (int i = tid; i < n; i += 128 * GROUPS)
        if (state(i)[S::H + c] != 0.0f) M = fmaxf(M, state(i)[c]);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if ((tid & 31) == 0) sm[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < GROUPS * 4; ++x) M = fmaxf(M, sm[x]);
    for (int i = tid; i < n; i += 128 * GROUPS) {
        const float l = state(i)[S::H + c];
        sw[i] = l == 0.0f ? 0.0f : ex2(state(i)[c] - M) * l;
    }
    __syncthreads();
    float o = 0.0f, w = 0.0f;
#pragma unroll
    for (int x = 0; x < kDeep; ++x)
        if (grp + x * GROUPS < n) {
            o = fmaf(sw[grp + x * GROUPS], v[x], o);
            w += sw[grp + x * GROUPS];
        }
#pragma unroll 8
    for (int i = grp + kDeep * GROUPS; i < n; i += GROUPS) {
        o = fmaf(sw[i], state(i)[2 * S::H + c * 128 + d], o);
        w += sw[i];
    }
    so[grp][d] = o;
    if (d == 0) sl[grp] = w;
    __syncthreads();
    if (grp == 0) {
        o = w = 0.0f;
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) {
            o += so[x][d];
            w += sl[x];
        }
        const int64_t at = (int64_t)item.x * p.Hq + (int64_t)item.y * S::H + c;
        o = w == 0.0f ? 0.0f : o / w;
        if (p.gate != nullptr && w != 0.0f) o = gated(p, at, o);
        p.out[at * 128 + d] = f32_to_bf16_bits(o);
    }
}

template <class S>
cudaError_t launch_shape(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int num_sms,
                         cudaStream_t stream, bool pdl) {
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        cudaError_t e1 = cudaFuncSetAttribute(paged_attn_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
        if (e1 != cudaSuccess) return e1;
        return cudaFuncSetAttribute(paged_attn_kernel<S>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    (int)cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms * S::kCtas < kPagedMaxCtas ? num_sms * S::kCtas : kPagedMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<S>, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    if (2 * p.N * p.G <= (int)cfg.gridDim.x) cfg.gridDim.x = (unsigned)(p.N * p.G);  // (the entries are by item then)
    cfg.gridDim.y = S::H;
    cfg.dynamicSmemBytes = 0;
    if ((int)(cfg.gridDim.x * cfg.gridDim.y) <= 2 * num_sms) {
        cfg.blockDim = dim3(128 * 8);
        return cudaLaunchKernelEx(&cfg, join_kernel<S, 8>, p);
    }
    cfg.blockDim = dim3(128 * 2);
    return cudaLaunchKernelEx(&cfg, join_kernel<S, 2>, p);
}

template <int H>
cudaError_t launch_heads(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int num_sms,
                         cudaStream_t stream, bool pdl) {
    if (p.sel_ids == nullptr) return launch_shape<Shape<H, false, false>>(p, kmap, vmap, num_sms, stream, pdl);
    if (H <= 8 && (int64_t)p.N * p.G >= 2 * num_sms)
        return launch_shape<Shape<H, true, H <= 8>>(p, kmap, vmap, num_sms, stream, pdl);
    return launch_shape<Shape<H, true, false>>(p, kmap, vmap, num_sms, stream, pdl);
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   int num_sms, cudaStream_t stream, bool pdl) {
    switch (p.Hq / p.G) {
        case 4: return launch_heads<4>(p, kmap, vmap, num_sms, stream, pdl);
        case 8: return launch_heads<8>(p, kmap, vmap, num_sms, stream, pdl);
        case 16: return launch_heads<16>(p, kmap, vmap, num_sms, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace step5
