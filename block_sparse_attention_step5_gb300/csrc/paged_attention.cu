// paged_attention.cu -- attention over the e4m3 paged cache on the tcgen05 tensor cores: every
// token of a causal window, or the picked regions plus the row's own.
//
//   s_t = softmax_scale (q . kcode_t) kscale(region of t),  p = softmax(s),  out = sum_t p_t vscale vcode_t
//
// The codes go to the tensor cores as they lie in the cache (kind::f8f6f4), so nothing is
// converted on the way and a key costs half the bytes of bf16.  The other operand of each product is then e4m3
// too, which has 4 significant bits; q and p are therefore split into parts, each the e4m3 rounding of
// what the parts before it left, times 2^5: two parts hold a bf16 q (8 bits) exactly down to 2^-22 of the
// head's largest value, three hold a weight to 12 bits, down to 2^-24 of the largest.  The parts are
// more columns of the small side of the product, which costs nothing at few heads: 128 keys are the M side,
//
//   S^T [128 keys x 2 H]  = K_tile [128 x 128 dims]       . (q parts)^T     (two TMEM buffers)
//   O^T [128 dims x 3 H] += V_tile^T [128 dims x 128 keys] . (p parts)^T
//
// with H query heads (of one row, or of R consecutive rows).  A region (8 tokens x 128 B) is one
// 128-byte-swizzle atom: K-major A for the first product, MN-major A for the second, from one TMA
// box (pages whose length allows it come in boxes of up to 16 regions).
//
// Scales.  kscale multiplies the fp32 score.  vscale joins the weight before it is split, relative to
// a power of two not below any vscale so far, so that the parts' range is spent on what a key adds to the
// output; the row sum takes the weight without it.
//
// Work.  The tiles of all (rows, group) items are laid end to end and every CTA takes an equal
// run of them, so a ragged batch, one long row and a chunk of many rows all fill the GPU; an item that
// several CTAs share is joined by the last of them to finish (in CTA order, so the bits do not depend
// on timing).
//
// Roles in a CTA: softmax warps (one thread per key of the tile and 16 head columns), a warp that issues
// the MMAs, two that issue the copies, K a tile ahead of V.
#include "paged.cuh"
#include "tcgen05.cuh"

namespace step5 {

namespace {

constexpr int kTile = 16;            // regions of a tile
constexpr int kLoadWarps = 2;
constexpr uint32_t kSlotBytes = kTile * 1024;
constexpr float kSlack = 3.0f;       // log2 units a tile's maximum may pass the running one by
constexpr float kPTop = 32.0f;       // weights are split from p * 2^(8 - slack): at most 2^8, whose parts fit e4m3
constexpr float kPart = 32.0f;       // a part against the one before it

template <int HQ_, int R_>
struct Shape {
    static constexpr int HQ = HQ_, R = R_, H = HQ * R;
    static constexpr int WG = H > 16 ? H / 16 : 1;     // softmax warpgroups
    static constexpr int C = H / WG;                   // head columns of a softmax thread
    static constexpr int RC = C / HQ;                  // rows of a softmax thread
    static constexpr int NS = 2 * H < 16 ? 16 : 2 * H;
    static constexpr int NO = (3 * H + 15) / 16 * 16;
    static constexpr int kSoft = WG * 128;
    static constexpr int kThreads = kSoft + 32 + 32 * kLoadWarps;
    static constexpr int kSlots = R > 1 ? 8 : (H > 8 ? 5 : 6);
    static constexpr int kCtas = R > 1 ? 1 : 2;        // per SM
    static constexpr uint32_t kCols = 2 * NS + NO <= 64 ? 64 : 2 * NS + NO <= 128 ? 128 : 2 * NS + NO <= 256 ? 256 : 512;
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

// Barrier over a named group of threads, returning whether any of them passed `v`.
__device__ __forceinline__ bool group_or(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

// Waits for phase `parity` of the barrier; gives up after 2^22 polls (far beyond any copy or product).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = smem_u32(bar);
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return false;
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The next part of two values: its codes, and what is left of the values times 2^5.
__device__ __forceinline__ uint32_t next_part(float& a, float& b) {
    const uint32_t c = e4m3x2(a, b);
    const float2 f = e4m3x2_to_f32x2((uint16_t)c);
    a = (a - f.x) * kPart;
    b = (b - f.y) * kPart;
    return c;
}

// The keys of a row: tokens lo .. pos of sequence b (b < 0: none).
struct Row {
    int b, pos, lo;
};

// Row n; b = -1 for padding and rows past N, -2 for a row out of range (which gets zeros).
__device__ __forceinline__ Row row_at(const PagedAttnParams& p, int n) {
    Row r{-1, -1, 0};
    if (n >= p.N) return r;
    r.b = p.row_seq[n];
    r.pos = p.row_pos[n];
    if (r.b == -1) return r;
    if (r.b < 0 || r.b >= p.B || r.pos < 0 || r.pos / p.pages.page_tokens >= p.pages.table_len) {
        r.b = -2;
        return r;
    }
    r.lo = p.window > 0 ? max(0, r.pos - p.window + 1) : 0;
    return r;
}

__device__ __forceinline__ int picks_of(const PagedAttnParams& p, int n, int g) {
    return min(max(p.sel_count[(int64_t)n * p.G + g], 0), p.top_k);
}

__device__ __forceinline__ int tiles_of(int lo, int pos, int k) {
    return ((pos >> 3) - ((lo >> 3) & ~(k - 1))) / kTile + 1;
}

// Tiles of item (group g, block of R rows), as one thread counts them: those of each
// sequence of the block in turn; one for a block that only has rows out of range.
template <int R>
__device__ __forceinline__ int item_tiles(const PagedAttnParams& p, int64_t item, int blocks) {
    const int g = (int)(item / blocks), n0 = (int)(item % blocks) * R;
    if constexpr (R == 1) {
        const Row r = row_at(p, n0);
        if (r.b == -1) return 0;
        if (r.b < 0) return 1;
        return p.sel_ids ? (picks_of(p, n0, g) + kTile) / kTile : tiles_of(r.lo, r.pos, p.box_regions);
    } else {
        int b[R], t = 0;
        bool any = false;
        for (int j = 0; j < R; ++j) b[j] = row_at(p, n0 + j).b;
        for (int j = 0; j < R; ++j) {
            any |= b[j] == -2;
            if (b[j] < 0) continue;
            int lo = INT32_MAX, hi = 0;
            const int mine = b[j];
            for (int i = j; i < R; ++i)
                if (b[i] == mine) {
                    const Row r = row_at(p, n0 + i);
                    lo = min(lo, r.lo);
                    hi = max(hi, r.pos);
                    b[i] = -1;
                }
            t += tiles_of(lo, hi, p.box_regions);
        }
        return t ? t : (any ? 1 : 0);
    }
}

// The tiles of an item as a warp walks them.  In a sequence's pass, tile i holds entries
// 16 i .. 16 i + 15: regions r0 + e of the sequence, or the e-th pick and the own region behind them.
template <int R>
struct Walk {
    Row mine;        // lane j < R: row j of the block
    uint32_t valid;  // its rows with keys
    uint32_t todo;   // not yet walked
    int n0, g;
    int b, lo, hi;   // this pass: the sequence, its first and last token
    uint32_t rows;   //   and the block's rows in it
    int r0, entries, tiles, at;  // first region, entries, tiles, tile in the pass
    const int32_t* ids;

    __device__ __forceinline__ int open(const PagedAttnParams& p, int64_t item, int blocks, int lane) {
        g = (int)(item / blocks);
        n0 = (int)(item % blocks) * R;
        mine = Row{-1, -1, 0};
        if (lane < R) mine = row_at(p, n0 + lane);
        valid = __ballot_sync(0xffffffffu, mine.b >= 0);
        const uint32_t bad = __ballot_sync(0xffffffffu, mine.b == -2);
        ids = p.sel_ids ? p.sel_ids + ((int64_t)n0 * p.G + g) * p.top_k : nullptr;
        todo = valid;
        int t = 0;
        while (todo) {
            pass(p);
            t += tiles;
        }
        todo = valid;
        if (valid == 0) {  // one empty tile if anything is to be written
            b = -1, rows = 0, r0 = 0, entries = 0, at = 0, lo = 0, hi = -1;
            tiles = bad ? 1 : 0;
            return tiles;
        }
        pass(p);
        return t;
    }
    __device__ __forceinline__ void pass(const PagedAttnParams& p) {
        const int lead = __ffs(todo) - 1;
        b = __shfl_sync(0xffffffffu, mine.b, lead);
        const bool in = mine.b == b;
        rows = __ballot_sync(0xffffffffu, in);
        todo &= ~rows;
        lo = __reduce_min_sync(0xffffffffu, in ? mine.lo : INT32_MAX);
        hi = __reduce_max_sync(0xffffffffu, in ? mine.pos : 0);
        at = 0;
        if (ids) {
            r0 = 0;
            entries = picks_of(p, n0, g) + 1;
            tiles = (entries + kTile - 1) / kTile;
        } else {
            r0 = (lo >> 3) & ~(p.box_regions - 1);
            entries = (hi >> 3) - r0 + 1;
            tiles = (entries + kTile - 1) / kTile;
        }
    }
    __device__ __forceinline__ void skip(const PagedAttnParams& p, int n) {  // to n tiles further on
        while (n >= tiles - at && todo) {
            n -= tiles - at;
            pass(p);
        }
        at += n;
    }
    // The region of entry q of the current tile, or -1.
    __device__ __forceinline__ int region(int q) const {
        const int e = at * kTile + q;
        if (b < 0 || e >= entries) return -1;
        if (!ids) return r0 + e;
        return e == entries - 1 ? hi >> 3 : __ldg(ids + e);
    }
};

// The pool row of a region's first token; -1 for a region that is none of the pass's, -2 for one that
// cannot be read.
template <int R>
__device__ __forceinline__ int region_row(const PagedAttnParams& p, const Walk<R>& w, int q, int r) {
    const int e = w.at * kTile + q;
    if (w.b < 0 || e >= w.entries) return -1;
    if (w.ids) {
        const int own = w.hi >> 3;
        if (r < 0 || r > own || (r == own) != (e == w.entries - 1)) return -2;
    }
    const int64_t row = page_row(p.pages, p.G, w.b, w.g, r * 8);
    return row < 0 ? -2 : (int)row;
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kCtas)
    paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      PagedAttnParams p) {
    constexpr int H = S::H, C = S::C, R = S::R, RC = S::RC, HQ = S::HQ, WG = S::WG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw, 1024);
    uint8_t* slots = smem;
    uint8_t* qt = smem + S::kSlots * kSlotBytes;
    uint8_t* pt = qt + S::kQBytes;
    __shared__ __align__(8) uint64_t full[S::kSlots], empty[S::kSlots], sbar[2], obar[2], pbar[2], qbar;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail, s_last;
    __shared__ int s_note[S::kSlots];  // of the item in a slot: MMA steps | first tile of a segment << 8 | last << 9
    __shared__ float red[WG][3][4][C + 1], s_cq[2][H];
    __shared__ int64_t s_scan[S::kThreads / 32], s_item;
    __shared__ int s_off;
    __shared__ uint32_t s_nan[R > 1 ? 128 : 1];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int blocks = (p.N + R - 1) / R;
    const int64_t items = (int64_t)blocks * p.G;
    constexpr int kMmaWarp = S::kSoft / 32, kLoadWarp = kMmaWarp + 1;

    if (tid == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        for (int s = 0; s < S::kSlots; ++s) {
            mbar_init(&full[s], kLoadWarps);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sbar[s], 1);
            mbar_init(&obar[s], 1);
            mbar_init(&pbar[s], S::kSoft);
        }
        mbar_init(&qbar, S::kSoft);
        fence_mbar_init();
        s_fail = 0;
    }
    if (warp == 0) tc::alloc(&s_tmem, S::kCols);
    if (2 * H < S::NS)  // q rows that no head fills
        for (int i = tid; i < (int)(S::NS - 2 * H) * 8; i += S::kThreads)
            reinterpret_cast<uint4*>(qt + 2 * H * 128)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_launch_dependents();

    // this CTA's run of tiles: thread sums of the items' tiles, their prefix, the item that the run starts in
    int64_t total, start, per;
    {
        const int64_t chunk = (items + S::kThreads - 1) / S::kThreads;
        const int64_t i0 = min(items, tid * chunk), i1 = min(items, i0 + chunk);
        int64_t sum = 0;
        for (int64_t i = i0; i < i1; ++i) sum += item_tiles<R>(p, i, blocks);
        int64_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int64_t before = inc - sum;
        total = 0;
        for (int w = 0; w < S::kThreads / 32; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        per = (total + gridDim.x - 1) / gridDim.x;
        if (per < p.min_tiles) per = p.min_tiles;
        start = blockIdx.x * per;
        if (start >= before && start < before + sum) {
            int64_t at = before;
            for (int64_t i = i0; i < i1; ++i) {
                const int t = item_tiles<R>(p, i, blocks);
                if (start < at + t) {
                    s_item = i;
                    s_off = (int)(start - at);
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
    const int run = (int)(start < total ? min(per, total - start) : 0);
    const int64_t item0 = s_item;
    const int off0 = s_off;

    if (run == 0) {
        // nothing to do
    } else if (warp >= kLoadWarp) {
        // ---------------- load warps: K_0, K_1, V_0, K_2, V_1, ... over the run's tiles, each into
        // the next slot once the product that read it is done.  Warp lw takes half of a tile's boxes.
        const int lw = warp - kLoadWarp;
        const int k = p.box_regions, boxes = kTile / k;
        const int half = boxes > 1 ? boxes / 2 : 1;
        const int q = (lw * half + lane) * k;  // first entry of this lane's box
        const bool has = lane < half && q < kTile;
        bool ok = true;
        int j = 0;  // slot uses so far
        Walk<R> w;
        int64_t item = item0;
        int left = run, in_seg = 0;      // tiles of the run, of the segment, not yet walked
        bool first = false;
        auto put = [&](bool isv, int row, int note, uint32_t zero) {
            const int slot = j % S::kSlots, use = j / S::kSlots;
            if (use > 0 && !wait(&empty[slot], (uint32_t)((use - 1) & 1))) ok = false;
            if (*reinterpret_cast<volatile int*>(&s_fail) != 0) ok = false;
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                return;
            }
            ++j;
            uint8_t* dst = slots + slot * kSlotBytes;
            // regions of V inside the product's steps that no copy fills
            const bool wrote = isv && zero != 0;
            if (wrote) {
                for (uint32_t z = zero; z; z &= z - 1) {
                    uint4* at = reinterpret_cast<uint4*>(dst + (__ffs(z) - 1) * 1024);
                    at[lane] = make_uint4(0, 0, 0, 0);
                    at[lane + 32] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
            }
            if (lw == 0 && lane == 0) s_note[slot] = note;
            const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)__popc(have) * 1024u * k);
            __syncwarp();
            if (row >= 0) tma_load_2d(dst + q * 1024, isv ? &vmap : &kmap, &full[slot], 0, row);
        };
        int row = -1, note = 0, nrow = -1, nnote = 0;  // the tile whose V is next, and the one after it
        uint32_t zero = 0, nzero = 0;
        int off = off0;
        for (int t = 0; t <= run && ok; ++t) {
            nrow = -1, nnote = 0, nzero = 0;
            if (t < run) {
                if (in_seg == 0) {  // the next segment
                    int nt = 0;
                    for (; item < items; ++item) {
                        nt = w.open(p, item, blocks, lane);
                        if (nt > off) break;
                    }
                    if (item >= items) {  // (the run counts other tiles than the rows have now)
                        ok = false;
                        break;
                    }
                    w.skip(p, off);
                    in_seg = min(nt - off, left);
                    left -= in_seg;
                    off = 0;
                    ++item;
                    first = true;
                } else if (w.at + 1 < w.tiles) {
                    ++w.at;
                } else {
                    w.pass(p);
                }
                --in_seg;
                // a box is copied when any of its regions is one of the pass's
                const int n_ent = w.b < 0 ? 0 : min(kTile, (w.entries - w.at * kTile + k - 1) / k * k);
                const int steps = (n_ent + 3) >> 2;
                if (has && q < n_ent) {
                    const int e = w.at * kTile + q;
                    int r = -1;
                    if (w.ids)
                        r = w.region(q);
                    else if (w.r0 + e + k > (w.lo >> 3))
                        r = w.r0 + e;
                    if (w.ids || r >= 0) nrow = region_row(p, w, q, r);
                    if (nrow == -2) raise_status(p.status, kDevRange);
                }
                // regions of the steps without a copy: by box, for both load warps' boxes alike
                const uint32_t got = __ballot_sync(0xffffffffu, nrow >= 0);
                const uint32_t mine = ((1u << (half * k)) - 1u) << (lw * half * k);
                uint32_t filled = 0;
                for (uint32_t b = got; b; b &= b - 1) filled |= ((1u << k) - 1u) << ((lw * half + __ffs(b) - 1) * k);
                nzero = lw * half * k < kTile ? ~filled & mine & ((1u << (4 * steps)) - 1u) : 0u;
                nnote = steps | (first ? 256 : 0) | (in_seg == 0 ? 512 : 0);
                first = false;
                put(false, nrow, nnote, 0);
            }
            if (t > 0 && ok) put(true, row, note, zero);
            row = nrow, note = nnote, zero = nzero;
        }
        if (!ok) {
            // a wait gave up: let the copies issued land (bounded) before the shared memory goes away
            if (lane == 0) {
                raise_status(p.status, kDevTimeout);
                atomicExch(&s_fail, 1);
                for (int i = (j > S::kSlots ? j - S::kSlots : 0); i < j; ++i)
                    wait(&full[i % S::kSlots], (uint32_t)((i / S::kSlots) & 1));
            }
            __syncwarp();
        }
    } else if (warp == kMmaWarp) {
        // ---------------- MMA warp: lane 0 issues both products of every tile
        const uint32_t slot_addr = smem_u32(slots), p_addr = smem_u32(pt);
        const uint64_t dq = tc::smem_desc(smem_u32(qt), 16, 1024, tc::kSwizzle128);
        bool ok = true;
        uint64_t* last_commit = nullptr;
        uint32_t last_parity = 0;
        int seg = 0;
        bool k_last = false;  // whether the tile whose first product was issued last ends its segment
        auto use = [&](int j, auto&& issue) {  // the product that reads the j-th slot use
            const int slot = j % S::kSlots;
            const uint32_t parity = (uint32_t)((j / S::kSlots) & 1);
            if (!ok || !__all_sync(0xffffffffu, wait(&full[slot], parity))) {
                ok = false;
                return;
            }
            const int note = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_note[slot]), 0);
            if (!issue(slot, note)) {
                ok = false;
                return;
            }
            last_commit = &empty[slot];
            last_parity = parity;
        };
        auto mma1 = [&](int t) {
            use(t == 0 ? 0 : 2 * t - 1, [&](int slot, int note) {
                k_last = (note & 512) != 0;
                if ((note & 256) && !__all_sync(0xffffffffu, wait(&qbar, (uint32_t)(seg++ & 1)))) return false;
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint64_t da = tc::smem_desc(slot_addr + slot * kSlotBytes, 16, 1024, tc::kSwizzle128);
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // 32 dims each
                        tc::mma_f8(tmem + (uint32_t)(S::NS * (t & 1)), da + 2 * i, dq + 2 * i, S::kIdesc1, i > 0);
                    tc::commit(&sbar[t & 1]);
                    tc::commit(&empty[slot]);
                }
                __syncwarp();
                return true;
            });
        };
        auto mma2 = [&](int t) {
            // K_t is use 2 t - 1, V_t use 2 t + 2 (one less for the last tile, which no K follows)
            use(t + 1 < run ? 2 * t + 2 : 2 * t + 1, [&](int slot, int note) {
                tc::fence_after_sync();
                if (lane == 0) {
                    const uint64_t da = tc::smem_desc(slot_addr + slot * kSlotBytes, 16, 1024, tc::kSwizzle128);
                    const uint64_t db = tc::smem_desc(p_addr + (uint32_t)(t & 1) * S::kPBytes, S::kPGroup, 128, tc::kSwizzleNone);
                    for (int i = 0; i < (note & 255); ++i)  // 32 keys (four regions) each
                        tc::mma_f8(tmem + 2u * S::NS, da + 256u * i, db + (uint32_t)(S::kPGroup >> 2) * i, S::kIdesc2,
                                   !(note & 256) || i > 0);
                    tc::commit(&obar[t & 1]);
                    tc::commit(&empty[slot]);
                }
                __syncwarp();
                return true;
            });
        };
        // the first product of the next tile goes ahead of the second of this one, except
        // behind a segment's last tile: its q replaces this segment's
        mma1(0);
        for (int t = 0; t < run && ok; ++t) {
            const bool last = k_last;
            if (t + 1 < run && !last) mma1(t + 1);
            if (ok && !wait(&pbar[t & 1], (uint32_t)((t >> 1) & 1))) ok = false;
            if (*reinterpret_cast<volatile int*>(&s_fail) != 0) ok = false;
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            mma2(t);
            if (t + 1 < run && last && ok) mma1(t + 1);
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
        // ---------------- softmax warps: one key per thread (its TMEM lane), C head columns
        const int wg = warp >> 2, key = tid & 127, q = key >> 3, c0 = wg * C, j0 = c0 / HQ;
        float m_ref[C], l_part[C], vref = 0.0f;
        // what the epilogue of the segment before needs of it
        int e_n0 = 0, e_g = 0, e_nt = 0, e_off = 0, e_seg = 0;
        int64_t e_begin = 0;
        uint32_t e_write = 0;
        bool failed = false;
        int t = 0;  // tile of the run

        // over all softmax warps, so that they give up together
        auto bar_or = [&](bool v) { return group_or(1, S::kSoft, v); };
        auto give_up = [&] {
            raise_status(p.status, kDevTimeout);
            atomicExch(&s_fail, 1);
        };
        auto gone = [&](bool w_ok) {
            if (!w_ok) give_up();
            return failed = bar_or(!w_ok || *reinterpret_cast<volatile int*>(&s_fail) != 0);
        };

        // The segment's heads as two e4m3 parts each: 16 lanes to a head.
        auto build_q = [&](const Walk<R>& w, float* cq) {
            for (int u = tid >> 4; u < H; u += S::kSoft / 16) {
                const int n = w.n0 + u / HQ, d8 = tid & 15;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (w.valid >> (u / HQ) & 1u)
                    x = *reinterpret_cast<const uint4*>(p.q + ((int64_t)n * p.Hq + (int64_t)w.g * HQ + u % HQ) * 128 + d8 * 8);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t a = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) a = max(a, max(xs[i] & 0x7fffu, (xs[i] >> 16) & 0x7fffu));
#pragma unroll
                for (int d = 8; d; d >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, d));
                const bool finite = a < 0x7f80u;
                // q * 2^(7 - e) lies in [2^7, 2^8) for the largest |q| = 2^e ..
                const int e = a == 0 ? 0 : max((int)(a >> 7) - 127, -100);
                const float up = __uint_as_float((uint32_t)(min(7 - e, 120) + 127) << 23);
                if (d8 == 0) cq[u] = finite ? p.scale_log2 / up : __int_as_float(0x7fc00000);
                uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f0 = bf16_lo(xs[i]) * up, f1 = bf16_hi(xs[i]) * up;
                    hi[i >> 1] |= next_part(f0, f1) << (16 * (i & 1));
                    lo[i >> 1] |= e4m3x2(f0, f1) << (16 * (i & 1));
                }
                auto at = [&](int r) {
                    return reinterpret_cast<uint2*>(qt + r * 128 + (((d8 >> 1) ^ (r & 7)) << 4) + (d8 & 1) * 8);
                };
                *at(u) = make_uint2(hi[0], hi[1]);
                *at(H + u) = make_uint2(lo[0], lo[1]);
            }
            fence_proxy_async();
            arrive(&qbar);
        };

        // O of the segment that ended with tile t - 1, and its output or partial state.
        auto epilogue = [&] {
            const int tl = t - 1;
            const bool w_ok = wait(&obar[tl & 1], (uint32_t)((tl >> 1) & 1));
            tc::fence_after_sync();
            float(&rd)[4][C + 1] = red[wg][2];
            int hidx = 0;
            const float sum = fold<C, 16>(l_part, lane, &hidx, Add{});
            if ((lane & (32 / C - 1)) == 0) rd[warp & 3][hidx] = sum;
            if (gone(w_ok)) return;  // (and every warpgroup's NaN notes are in before any is read)
            float o[C], L[C];
            const uint32_t ob = tc::taddr(tmem, (warp & 3) * 32, 2 * S::NS);
            if constexpr (C == 16) {
                float a[16], b[16];
                tc::ld16(ob + c0, o);
                tc::ld16(ob + H + c0, a);
                tc::ld16(ob + 2 * H + c0, b);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] += (a[c] + b[c] * (1.0f / kPart)) * (1.0f / kPart);
            } else {
                float a[16], b[16];
                tc::ld16(ob, a);
                if constexpr (C == 8) tc::ld16(ob + 16, b);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    o[c] = a[c] + (a[C + c] + (C == 8 ? b[c] : a[(2 * C + c) & 15]) * (1.0f / kPart)) * (1.0f / kPart);
            }
            const uint32_t nan = R > 1 ? s_nan[R > 1 ? key : 0] : 0u;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                L[c] = (rd[0][c] + rd[1][c]) + (rd[2][c] + rd[3][c]);
                o[c] = L[c] == 0.0f ? 0.0f : o[c] / L[c] * (vref * (1.0f / kPTop));
                if (R > 1 && (nan >> (j0 + c / HQ) & 1u)) o[c] = __int_as_float(0x7fc00000);
            }
            auto write = [&](int c, float v) {
                const int n = e_n0 + j0 + c / HQ;
                const int64_t h = (int64_t)n * p.Hq + (int64_t)e_g * HQ + c % HQ;
                if (!(e_write >> (j0 + c / HQ) & 1u)) return;
                if (p.gate != nullptr) v *= 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[h])));
                p.out[h * 128 + key] = f32_to_bf16_bits(v);
            };
            if (e_seg == e_nt) {
#pragma unroll
                for (int c = 0; c < C; ++c) write(c, o[c]);
            } else {
                // CTAs first .. last share the item; each leaves its state, the last to arrive joins them in order
                const int first = (int)(e_begin / per), last = (int)((e_begin + e_nt - 1) / per);
                auto state = [&](int cta) { return p.states + ((int64_t)2 * cta + (cta == first ? 1 : 0)) * S::kState; };
                float* st = state(blockIdx.x);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (key == 0) {
                        __stcg(st + c0 + c, m_ref[c]);
                        __stcg(st + H + c0 + c, L[c]);
                    }
                    __stcg(st + 2 * H + (c0 + c) * 128 + key, o[c]);
                }
                __threadfence();
                bar_or(false);
                if (tid == 0) {
                    const uint32_t n = (uint32_t)(last - first);
                    s_last = atomicInc(p.counters + first, n) == n;
                    __threadfence();
                }
                if (bar_or(tid == 0 && s_last != 0)) {
                    float M[C], W[C], O[C];
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        M[c] = -INFINITY;
                        W[c] = O[c] = 0.0f;
                    }
                    for (int i = first; i <= last; ++i) {
                        const float* si = state(i);
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            const float m = __ldcg(si + c0 + c), l = __ldcg(si + H + c0 + c);
                            const float v = __ldcg(si + 2 * H + (c0 + c) * 128 + key);
                            if (l == 0.0f) continue;
                            const float mn = fmaxf(M[c], m);
                            const float a = exp2f(M[c] - mn), b = exp2f(m - mn) * l;
                            M[c] = mn;
                            W[c] = W[c] * a + b;
                            O[c] = O[c] * a + b * v;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c) write(c, W[c] == 0.0f ? 0.0f : O[c] / W[c]);
                }
            }
            if (R > 1) {
                bar_or(false);
                if (tid < 128) s_nan[R > 1 ? tid : 0] = 0;
                bar_or(false);
            }
        };

        if (R > 1 && tid < 128) s_nan[R > 1 ? tid : 0] = 0;

        Walk<R> w;
        int64_t item = item0;
        int off = off0;
        int segs = 0;
        for (int left = run; left > 0; ++item) {
            if (item >= items) {
                give_up();
                failed = true;
                break;
            }
            const int nt = w.open(p, item, blocks, lane);
            if (nt <= off) continue;
            float* cq = s_cq[segs++ & 1];
            build_q(w, cq);
            if (warp == 0) {
                if (w.mine.b == -2) raise_status(p.status, kDevRange);
                if (p.sel_ids && lane == 0 && w.valid) {
                    const int n = p.sel_count[(int64_t)w.n0 * p.G + w.g];
                    if (n < 0 || n > p.top_k) raise_status(p.status, kDevRange);
                }
            }
            if (t > 0)
                epilogue();
            else
                bar_or(false);
            if (failed) break;
            const int seg = min(nt - off, left);
            w.skip(p, off);
            e_n0 = w.n0, e_g = w.g, e_nt = nt, e_off = off, e_seg = seg;
            e_begin = start + (run - left) - off;
            e_write = __ballot_sync(0xffffffffu, w.mine.b != -1);
            left -= seg;
            off = 0;
            vref = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                m_ref[c] = -INFINITY;
                l_part[c] = 0.0f;
            }
            int row_lo[RC], row_pos[RC];
#pragma unroll
            for (int i = 0; i < RC; ++i) {
                row_lo[i] = __shfl_sync(0xffffffffu, w.mine.lo, j0 + i);
                row_pos[i] = __shfl_sync(0xffffffffu, w.mine.pos, j0 + i);
            }
            // lane l looks up entry 4 (warp % 4) + l % 4 of tile l / 4 of the next eight: its pool row and scales
            int b_row = -1;
            float b_ks = 0.0f, b_vs = 0.0f;
            int batch = -1;
            for (int i = 0; i < seg; ++i, ++t) {
                if (i > 0) {
                    if (w.at + 1 < w.tiles) {
                        ++w.at;
                    } else {
                        w.pass(p);
                        batch = -1;
                    }
                }
                if (batch != w.at >> 3) {
                    batch = w.at >> 3;
                    Walk<R> v = w;
                    v.at = batch * 8 + (lane >> 2);
                    const int qe = 4 * (warp & 3) + (lane & 3), e = v.at * kTile + qe, k = p.box_regions;
                    b_row = -1;
                    int r = -1;
                    if (w.ids) {
                        if (e < w.entries) {
                            r = v.region(qe);
                            b_row = region_row(p, v, qe, r);
                        }
                    } else if (w.b >= 0 && e < (w.entries + k - 1) / k * k && ((w.r0 + e) | (k - 1)) >= (w.lo >> 3)) {
                        r = w.r0 + e;
                        const int64_t at = page_row(p.pages, p.G, w.b, w.g, r * 8);
                        b_row = at < 0 ? -2 : (int)at;
                    }
                    b_ks = b_vs = 0.0f;
                    if (b_row >= 0) {
                        b_ks = __ldg(p.k_scales + (b_row >> 3));
                        b_vs = __ldg(p.v_scales + (b_row >> 3));
                        if (!scale_ok(b_ks) || !scale_ok(b_vs)) {
                            if (w.ids || (r >= (w.lo >> 3) && r <= (w.hi >> 3))) raise_status(p.status, kDevRange);
                            b_ks = 0.0f;
                        }
                    }
                }
                const int from = (w.at & 7) * 4 + (lane >> 3);
                const bool loaded = __shfl_sync(0xffffffffu, b_row, from) >= 0;
                const float ks = __shfl_sync(0xffffffffu, b_ks, from), vs = __shfl_sync(0xffffffffu, b_vs, from);
                const int e = w.at * kTile + q;
                const bool own = w.ids && e == w.entries - 1;
                const int tok = (w.ids ? (own ? w.hi >> 3 : 0) : w.r0 + e) * 8 + (key & 7);
                const bool readable = loaded && ks > 0.0f && tok >= w.lo && tok <= w.hi;
                bool sees[RC];
#pragma unroll
                for (int r = 0; r < RC; ++r)
                    sees[r] = readable && (R == 1 || ((w.rows >> (j0 + r) & 1u) && tok >= row_lo[r] && tok <= row_pos[r]));

                bool w_ok = wait(&sbar[t & 1], (uint32_t)((t >> 1) & 1));
                tc::fence_after_sync();
                float s[C];
                const uint32_t sb = tc::taddr(tmem, (warp & 3) * 32, (uint32_t)(S::NS * (t & 1)));
                if constexpr (C == 16) {
                    float lo[16];
                    tc::ld16(sb + c0, s);
                    tc::ld16(sb + H + c0, lo);
#pragma unroll
                    for (int c = 0; c < C; ++c) s[c] = fmaf(lo[c], 1.0f / kPart, s[c]);
                } else {
                    float x[16];
                    tc::ld16(sb, x);
#pragma unroll
                    for (int c = 0; c < C; ++c) s[c] = fmaf(x[C + c], 1.0f / kPart, x[c]);
                }
                float mx[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    s[c] = sees[c / HQ] ? s[c] * (cq[c0 + c] * ks) : -INFINITY;
                    mx[c] = s[c];
                }
                int hidx = 0;
                const float wmax = fold<C, 16>(mx, lane, &hidx, Max{});
                const uint32_t vmax = __reduce_max_sync(0xffffffffu, readable ? __float_as_uint(vs) : 0u);
                float(&rd)[4][C + 1] = red[wg][t & 1];
                if ((lane & (32 / C - 1)) == 0) rd[warp & 3][hidx] = wmax;
                if (lane == 0) rd[warp & 3][C] = __uint_as_float(vmax);
                if (gone(w_ok)) break;
                // the running maxima move when a tile's passes them by more than the slack, vref when a
                // tile's vscale passes it; then l and O are rescaled.  Every thread of the warpgroup does the same.
                bool move = false;
                float ratio = 1.0f;
                {
                    const float v = fmaxf(fmaxf(rd[0][C], rd[1][C]), fmaxf(rd[2][C], rd[3][C]));
                    if (v > vref) {
                        const uint32_t u = __float_as_uint(v);
                        const float next = __uint_as_float((u & 0x7f800000u) + ((u & 0x7fffffu) ? 0x800000u : 0u));
                        ratio = vref / next;
                        vref = next;
                        move = true;
                    }
                }
                float alpha[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float tmax = fmaxf(fmaxf(rd[0][c], rd[1][c]), fmaxf(rd[2][c], rd[3][c]));
                    alpha[c] = 1.0f;
                    if (tmax > m_ref[c] + kSlack || (m_ref[c] == -INFINITY && tmax > -INFINITY)) {
                        alpha[c] = exp2f(m_ref[c] - tmax);
                        m_ref[c] = tmax;
                        move = true;
                    }
                }
                const float vf = vref > 0.0f ? vs * (1.0f / vref) * kPTop : 0.0f;
                float w8[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float pv = s[c] == -INFINITY ? 0.0f : exp2f(s[c] - m_ref[c]);
                    l_part[c] = l_part[c] * alpha[c] + pv;
                    w8[c] = pv * vf;
                }
                // the P buffer was last read by the second product two tiles back
                if (t >= 2) w_ok &= wait(&obar[t & 1], (uint32_t)(((t >> 1) - 1) & 1));
                {
                    uint32_t part[3][C / 4];
#pragma unroll
                    for (int c = 0; c < C; c += 4) {
                        float a = w8[c], b = w8[c + 1], d = w8[c + 2], f = w8[c + 3];
                        part[0][c / 4] = next_part(a, b) | (next_part(d, f) << 16);
                        part[1][c / 4] = next_part(a, b) | (next_part(d, f) << 16);
                        part[2][c / 4] = e4m3x2(a, b) | (e4m3x2(d, f) << 16);
                    }
                    uint8_t* pb = pt + (t & 1) * S::kPBytes + q * S::kPGroup + (key & 7) * 16;
                    if constexpr (C == 16) {
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            *reinterpret_cast<uint4*>(pb + (i * H + c0) * 8) =
                                make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
                    } else if constexpr (C == 8) {
                        *reinterpret_cast<uint4*>(pb) = make_uint4(part[0][0], part[0][1], part[1][0], part[1][1]);
                        *reinterpret_cast<uint4*>(pb + 128) = make_uint4(part[2][0], part[2][1], 0u, 0u);
                    } else {
                        *reinterpret_cast<uint4*>(pb) = make_uint4(part[0][0], part[1][0], part[2][0], 0u);
                    }
                }
                if (move && i > 0) {
                    w_ok &= wait(&obar[(t - 1) & 1], (uint32_t)(((t - 1) >> 1) & 1));
                    tc::fence_after_sync();
                    const uint32_t ob = tc::taddr(tmem, (warp & 3) * 32, 2 * S::NS);
#pragma unroll
                    for (int i16 = 0; i16 < (C == 16 ? 3 : S::NO / 16); ++i16) {
                        const uint32_t at = ob + (C == 16 ? i16 * H + c0 : i16 * 16);
                        float o[16];
                        tc::ld16(at, o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] *= alpha[c % C] * ratio;
                        tc::st16(at, o);
                    }
                }
                // V rows of keys that no row of the block sees are zeroed (the cache may hold anything
                // there and a zero weight must meet a finite value); of keys that some rows do
                // not see, NaN codes are taken out and noted for the rows that do
                if (wg == 0) {
                    uint32_t seen = readable ? w.valid : 0u;  // the rows that see this key
                    if constexpr (R > 1) {
                        const bool in = w.rows >> lane & 1u;
                        const int max_lo = __reduce_max_sync(0xffffffffu, in ? w.mine.lo : 0);
                        const int min_pos = __reduce_min_sync(0xffffffffu, in ? w.mine.pos : INT32_MAX);
                        const int t0 = (w.r0 + w.at * kTile) * 8;
                        if (w.rows != w.valid || t0 < max_lo || t0 + kTile * 8 - 1 > min_pos) {
                            seen = 0;
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                const int lo = __shfl_sync(0xffffffffu, w.mine.lo, r), pos = __shfl_sync(0xffffffffu, w.mine.pos, r);
                                if (readable && (w.rows >> r & 1u) && tok >= lo && tok <= pos) seen |= 1u << r;
                            }
                        }
                    }
                    if (loaded && seen != w.valid) {
                        const int jv = t + 1 < run ? 2 * t + 2 : 2 * t + 1, slot = jv % S::kSlots;
                        w_ok &= wait(&full[slot], (uint32_t)((jv / S::kSlots) & 1));
                        uint32_t* vr = reinterpret_cast<uint32_t*>(slots + slot * kSlotBytes + key * 128);
                        if (seen == 0) {
#pragma unroll
                            for (int x = 0; x < 8; ++x) reinterpret_cast<uint4*>(vr)[x] = make_uint4(0, 0, 0, 0);
                        } else if constexpr (R > 1) {
                            for (int x = 0; x < 32; ++x) {
                                const uint32_t c = vr[x];
                                // bytes 0x7f and 0xff
                                uint32_t bad = ((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                if (bad == 0) continue;
                                vr[x] = c & ~((bad >> 7) * 0xffu);
                                const int d = (((x >> 2) ^ (key & 7)) << 4) + (x & 3) * 4;
                                for (; bad; bad &= bad - 1) atomicOr(&s_nan[d + ((__ffs(bad) - 1) >> 3)], seen);
                            }
                        }
                    }
                }
                fence_proxy_async();
                tc::fence_before_sync();
                if (!w_ok) give_up();  // (the warps leave together at the next barrier)
                arrive(&pbar[t & 1]);
            }
            if (failed) break;
        }
        if (!failed) epilogue();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) tc::dealloc(tmem, S::kCols);
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
    const int most = kPagedMaxCtas / (S::R > 1 ? 2 : 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms * S::kCtas < most ? num_sms * S::kCtas : most));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, paged_attn_kernel<S>, kmap, vmap, p);
}

template <int HQ>
cudaError_t launch_heads(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int num_sms,
                         cudaStream_t stream, bool pdl) {
    // rows of one sequence share its tiles when the sequences have two or more on average
    if (p.sel_ids == nullptr && p.N >= 2 * p.B)
        return launch_shape<Shape<HQ, 64 / HQ>>(p, kmap, vmap, num_sms, stream, pdl);
    return launch_shape<Shape<HQ, 1>>(p, kmap, vmap, num_sms, stream, pdl);
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
