// paged_attention_bf16.cu -- attention over the bf16 paged cache for few rows a sequence: every token of a causal window,
// or the picked regions plus the row's own.
//
//   s_t = softmax_scale (q . k_t),  p = softmax(s),  out = sum_t p_t v_t
//
// As over the e4m3 pages, 128 keys are the M side of both products, and the C columns of an item the small one: the H heads of R
// rows (1, or 2 or 4 neighbouring rows of the call, which mostly are one sequence's drafts and read its keys once),
//
//   S^T [128 keys x C]    = K_tile [128 x 128 dims]        . q^T            (two TMEM buffers)
//   O^T [128 dims x 2 C] += V_tile^T [128 dims x 128 keys] . (p parts)^T
//
// with bf16 operands as the cache has them.  A weight has 8 bits in bf16; what its first part leaves goes along as a second part, more columns of
// the small side, which cost nothing, so 16 bits of each weight meet V.  A region (8 tokens x 256 B) lands as two swizzle atoms,
// [half of the dims][8 tokens][128 B], from one box of a 4-D view of the pool (64 dims x 8 tokens x 2 halves x regions): the K-major
// operand of the first product and the MN-major one of the second.
//
// An item of several rows walks the keys of each of its sequences in turn, the other rows masked.  A weight of zero must meet a
// finite value: a V row that no row sees is zeroed, and where some rows see it and others do not, what is not finite in it is
// cleared and the token noted; the rows that see it take it up again from the page at their end.
//
// The split of the work, the roles of the warps and the join are those of the kernel over the e4m3 pages.  A tile is 64 KB, so one
// CTA an SM with 5 or 6 half tiles in shared memory, or two with 3, keep HBM busy; picks, whose copies are 2 KB each, want two CTAs
// (a CTA's copies of that size come at 44 GB/s out of L2, two CTAs' at 87).
//
// What bounds it, with 4 KV groups of 8 heads and pages of 64 tokens (by graph replay or call after call, join included):
//   one row of 4,608 tokens      9.2 us  latency: split, page and key loads, one tile, second product and states, join
//   16 rows of 16K to 32K        120 to 135 us (by lengths and GPU)  806 MB, 6.0 to 6.7 TB/s: HBM
//   8 x 4 rows behind 6K to 8K    31 us  117 MB in copies of 2 KB (pages of 24 tokens), 1.5 us a tile at their rate, start and join
//   one row of 512 picks         9.6 us  latency, as the short row
//   16 rows of 512 picks          29 us  start and join (10 us), and 135 MB in copies of 2 KB out of HBM (1,024 picks 50 us, 2,048 88: 6.7 to 7 TB/s)
//   2,048 rows of 512 picks    1,298 us  17.2 GB of copies of 2 KB out of L2, 13.2 TB/s of the 13.7 that L2 gives copies of any size
#include "paged_items.cuh"

namespace step5 {

namespace {

constexpr int kSoft = 128;           // softmax threads
constexpr int kThreads = kSoft + 64 + 64;
constexpr int kQkWarp = 4, kLoadWarp = 6, kLoadWarps = 2;  // (the second product's warp is 5)
constexpr int kRing = 8;             // tiles whose masks are in shared memory
constexpr uint32_t kRegionBytes = 2048, kSlotBytes = kTile * kRegionBytes;
constexpr float kSlack = 8.0f;       // log2 units a tile's maximum may pass the running one by

constexpr float kNone = 3.0e38f;     // less the running maximum of a head without keys so far (finite: scores may be -infinity)

template <int H_, int R_, bool PICKS_, int CTAS_>
struct Shape {
    static constexpr int H = H_, R = R_, C = H * R;    // query heads of a group, rows of an item, columns: heads of row after row
    static constexpr bool PICKS = PICKS_;
    static constexpr int kCtas = CTAS_;                // per SM
    static constexpr int kSlots = CTAS_ == 2 ? 3 : C == 32 ? 5 : 6;
    static_assert(kSlots <= 6, "the barriers of copies and the ring are reused after 4 and 8 tiles");
    static constexpr int NS = C < 16 ? 16 : C;         // columns of S
    static constexpr int NO = 2 * C < 16 ? 16 : 2 * C; // columns of O: the weights' two parts
    static constexpr uint32_t kCols = 2 * NS + NO <= 64 ? 64 : 128;
    static constexpr uint32_t kQBytes = NS * 256, kPBytes = 128 * NO * 2;
    static constexpr uint32_t kPGroup = 16 * NO;       // bytes of 8 keys of P
    static constexpr uint32_t kSmem = 1024 + kSlots * kSlotBytes + kQBytes + 2 * kPBytes;
    static constexpr uint32_t kIdesc1 = tc::instr_desc(tc::kFmtBF16, false, false, 128, NS);
    static constexpr uint32_t kIdesc2 = tc::instr_desc(tc::kFmtBF16, true, true, 128, NO);
    static constexpr int kState = C * 130;             // floats of a partial state: m[C], l[C], o[C][128]
    static_assert(2 * NS + NO <= (int)kCols, "tensor memory");
    static_assert((size_t)kPagedMaxCtas * 2 * kState <= kPagedStateFloats, "workspace");
    static_assert(C <= 32 && (R == 1 || !PICKS), "columns; picks are a row's own");
};

// What a tile's softmax and second product need to know of it: product steps, and ...
enum : int { kFirst = 256, kRowsShift = 16 };  // the segment's first tile; the item's rows that its sequence is of

// The sum of what is not finite in dim `key` among tokens from .. to of sequence b, in the noted runs of 128 (0: nothing); a warp has
// 32 dims, and looks through 32 tokens at a time, a token a lane.  Rarely run, and apart from the code that is: 304 items of two
// rows of 16,000 tokens, such values at both ends, 1.71 ms where the call without them takes 1.58 (token after token: 39).
__device__ __noinline__ float not_finite(const PagedAttnParams& p, int b, int g, int key, int from, int to, unsigned long long runs) {
    const int lane = key & 31;
    const uint16_t* values = reinterpret_cast<const uint16_t*>(p.v_pages);
    float sum = 0.0f;
    for (uint32_t t0 = (uint32_t)from & ~31u; from <= to && t0 <= (uint32_t)to; t0 += 32) {
        if (!(runs >> (t0 >> 7 & 63) & 1u)) {
            t0 |= 96;
            continue;
        }
        const uint32_t t = t0 + lane;
        const int64_t row = t >= (uint32_t)from && t <= (uint32_t)to ? page_row(p.pages, p.G, b, g, (int)t) : -1;
        uint32_t any = 0;
        if (row >= 0) {
            const uint4* v = reinterpret_cast<const uint4*>(values + row * 128 + (key & ~31));
            auto all_ones = [](uint32_t u) { return ((u & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; };  // an exponent of all ones
#pragma unroll
            for (int i = 0; i < 4; ++i) any |= all_ones(v[i].x) | all_ones(v[i].y) | all_ones(v[i].z) | all_ones(v[i].w);
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, any != 0); m; m &= m - 1) {
            const float v = bf16_to_f32(values[__shfl_sync(0xffffffffu, row, __ffs(m) - 1) * 128 + key]);
            if (!(fabsf(v) < INFINITY)) sum += v;
        }
    }
    return sum;
}

template <class S>
__global__ void __launch_bounds__(kThreads, S::kCtas)
    paged_attn_bf16_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      PagedAttnParams p) {
    constexpr int H = S::H, R = S::R, C = S::C;
    constexpr bool PICKS = S::PICKS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw, 1024);
    uint8_t* slots = smem;
    uint8_t* qt = smem + S::kSlots * kSlotBytes;
    uint8_t* pt = qt + S::kQBytes;
    __shared__ __align__(8) uint64_t kfull[4], vfull[4], empty[S::kSlots], sbar[2], obar[2], pbar[2], qbar;
    __shared__ uint32_t ring[kRing][kTile];  // of a region: its tokens that the row sees | 256 if a copy brings it
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    __shared__ int s_note[kRing], s_t0[kRing];  // of a tile: product steps | kFirst | rows; (several rows) first token
    __shared__ float red[3][4][C], s_factor[C];  // s_factor: a column's gate over its sum, 0 without keys
    // Of segment i % 2 (several rows): first and last token whose values were cleared, and of which runs of 128 tokens such are (bit: the
    // run's number modulo 64).
    __shared__ int2 s_cleared[2];
    __shared__ unsigned long long s_runs[2];
    __shared__ RunSmem<kThreads> rs;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int items = (p.N + R - 1) / R * p.G;

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
    if (C < S::NS)  // q rows that no head fills (softmax threads, which fence them below)
        for (int i = tid; i < (S::NS - C) * 16; i += kSoft)
            if (tid < kSoft) {
                constexpr int n = C < S::NS ? (S::NS - C) * 8 : 1;
                const int half = i / n, r = i % n;
                reinterpret_cast<uint4*>(qt + half * S::NS * 128 + C * 128)[r] = make_uint4(0, 0, 0, 0);
            }
    pdl_wait();
    pdl_launch_dependents();

    int64_t start, per;
    const bool few = take_run<PICKS, kThreads, R>(p, rs, start, per);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const int run = rs.run, item0 = rs.item, off0 = rs.off;

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
        // Lane l looks up its entry in tile l / 8 of four tiles, in two steps (region; pool row), the
        // next four while these go by.
        int b_r = 0, b_row = -1, n_r = 0, n_row = -1, batch = -1, done = 0;
        const int32_t* ids = nullptr;
        RowSet<R> set{};                 // (several rows) the item's, its sequences not yet walked, and this one
        uint32_t todo = 0, rows = 1;
        auto look = [&](int of, int steps) {
            const int e = (of * 4 + (lane >> 3)) * kTile + q;
            if (steps & 1) {
                n_r = -1;
                if (PICKS) {
                    if (e < it.entries) n_r = e == it.entries - 1 ? it.hi >> 3 : ids[e];
                } else if constexpr (R > 1) {  // with its box, of which some region is a row's (windows may leave gaps)
                    const int z = it.r0 + e, t0 = (z & ~(k - 1)) * 8;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (it.b >= 0 && (rows >> r & 1u) && t0 <= set.pos[r] && (p.window == 0 || t0 + 8 * k > set.pos[r] - p.window + 1))
                            n_r = z;
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
                    uint4* to = reinterpret_cast<uint4*>(dst + (__ffs(z) - 1) * kRegionBytes);
#pragma unroll
                    for (int x = 0; x < 4; ++x) to[lane + 32 * x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
            }
            uint64_t* full = isv ? &vfull[t & 3] : &kfull[t & 3];
            const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) expect_tx(full, (uint32_t)__popc(have) * kRegionBytes * k);
            __syncwarp();
            if (row >= 0) tma_load_4d(dst + q * kRegionBytes, isv ? &vmap : &kmap, full, 0, 0, 0, row >> 3);
            if (!isv) {
                // (this slot was free, so the softmax is past tile t - 5 and the ring's entry is free too)
                if (lane >> 3 == (at & 3)) {
                    // (several rows: which tokens a row sees is the softmax's business)
                    const int t0 = b_r * 8;
                    const int a = min(max(it.lo - t0, 0), 8), z = min(max(it.hi - t0 + 1, 0), 8);
                    const uint32_t mask = b_row >= 0 && z > a ? ((1u << z) - 1u) & ~((1u << a) - 1u) : 0u;
                    ring[t & (kRing - 1)][q] = mask | (b_row >= 0 ? 256u : 0u);
                }
                if (lw == 0 && lane == 0) {
                    s_note[t & (kRing - 1)] = note;
                    if (R > 1) s_t0[t & (kRing - 1)] = (it.r0 + at * kTile) * 8;
                }
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
                    it = rs.it;
                    if (t > 0) {
                        it.tiles = 0;
                        while (nitem < items && (it = item_of<PICKS, R>(p, nitem)).tiles <= off) ++nitem;
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
                    if constexpr (R > 1) {
                        set = rows_at<R>(p, it.n);
                        todo = rows_with_keys(set);
                        it.tiles = 0;  // (from here on those of the sequence)
                    }
                } else {
                    ++at;
                }
                if constexpr (R > 1)
                    while (at >= it.tiles && todo) {  // the item's next sequence
                        at -= it.tiles;
                        const Pass a = next_pass<R>(p, set, todo);
                        it.b = a.b, it.lo = a.lo, it.hi = a.hi, it.r0 = a.r0, it.entries = a.entries, it.tiles = a.tiles;
                        rows = a.rows;
                        batch = -1, done = 0;
                    }
                --in_seg;
                if (batch != at >> 2) {
                    if (done != 3) look(at >> 2, 3 & ~done);
                    batch = at >> 2;
                    b_r = n_r, b_row = n_row, done = 0;
                } else if ((batch + 1) * 4 < it.tiles) {
                    const int todo = ((1 << (at & 3)) - 1) & 3 & ~done;  // one more step at tiles 1 and 2
                    look(batch + 1, todo);
                    done |= todo;
                }
                nrow = __shfl_sync(0xffffffffu, b_row, (at & 3) * 8 + (lane & 7));
                const uint32_t got = __ballot_sync(0xffffffffu, lane < 8 && nrow >= 0) & 0xffu;
                if (!boxes) nrow = -1;
                const int steps = it.b < 0 ? 0 : min(8, (it.entries - at * kTile + 1) >> 1);
                // a box of several regions is copied whole or not at all; every entry of it has its row
                nzero = (~got << (lw * 8)) & (0xffu << (lw * 8)) & ((1u << (2 * steps)) - 1u);
                nnote = steps | (first ? kFirst : 0) | (int)rows << kRowsShift;
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
                if ((note & kFirst) && !wait(&qbar, (uint32_t)(seg++ & 1))) ok = false;
            } else {
                if (!wait(&pbar[t & 1], (uint32_t)((t >> 1) & 1))) ok = false;
            }
            if (*reinterpret_cast<volatile int*>(&s_fail) != 0) ok = false;
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc::fence_after_sync();
            if (qk) {
                const uint64_t da = tc::smem_desc(slot_addr + slot * kSlotBytes, 16, kRegionBytes, tc::kSwizzle128);
                if (elect()) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 dims each
                        tc::mma_f16(tmem + (uint32_t)(S::NS * (t & 1)), da + (i < 4 ? 2 * i : 64 + 2 * (i - 4)),
                                    dq + (i < 4 ? 2 * i : S::NS * 8 + 2 * (i - 4)), S::kIdesc1, i > 0);
                    arrive(&sbar[t & 1]);  // (hands the tile's ring entry on, which came with its K)
                    tc::commit(&sbar[t & 1]);
                    tc::commit(&empty[slot]);
                }
            } else {
                const uint64_t da = tc::smem_desc(slot_addr + slot * kSlotBytes, 1024, kRegionBytes, tc::kSwizzle128);
                const uint64_t db = tc::smem_desc(p_addr + (uint32_t)(t & 1) * S::kPBytes, S::kPGroup, 128, tc::kSwizzleNone);
                if (elect()) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)  // 16 keys (two regions) each
                        if (i < (note & 255))
                            tc::mma_f16(tmem + 2u * S::NS, da + (2u * kRegionBytes >> 4) * i, db + (S::kPGroup >> 3) * i, S::kIdesc2,
                                        !(note & kFirst) || i > 0);
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
        float2 neg_m[C / 2], l_part[C / 2];  // less the running maxima, the row sums of this thread's keys
        Item it{}, done{};  // the segment's item; that of the segment before, for its epilogue
        int64_t done_begin = 0;
        RowSet<R> set{}, done_set{};     // (several rows) theirs
        int segs = 0;
        bool whole = true, begins = true;  // it has the whole item, its first tile
        bool failed = false;
        int t = 0;  // tile of the run

        auto give_up = [&] {
            raise_status(p.status, kDevTimeout);
            atomicExch(&s_fail, 1);
        };

        // The item's columns, 16 lanes to each.
        auto build_q = [&] {
#pragma unroll
            for (int u0 = 0; u0 < C; u0 += 8) {
                const int u = u0 + (tid >> 4), d8 = tid & 15;
                if (C < 8 && u >= C) break;  // (whole warps)
                uint4 x = make_uint4(0, 0, 0, 0);
                bool there = it.b >= 0;
                if constexpr (R > 1) there = (rows_with_keys(set) >> (u / H) & 1u) != 0;
                if (there)
                    x = *reinterpret_cast<const uint4*>(p.q + (int64_t)(it.n + u / H) * p.q_stride + ((int64_t)it.g * H + u % H) * 128 + d8 * 8);
                *reinterpret_cast<uint4*>(qt + (d8 >> 3) * S::NS * 128 + u * 128 + (((d8 & 7) ^ (u & 7)) << 4)) = x;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(&qbar);
        };

        // O of the segment that ended with tile t - 1, and its output or partial state.
        auto epilogue = [&] {
            const int tl = t - 1;
            float(&rd)[4][C] = red[2];
            int cidx = 0;
            float l[C];
#pragma unroll
            for (int c = 0; c < C; ++c) l[c] = c & 1 ? l_part[c / 2].y : l_part[c / 2].x;
            const float sum = fold<C, 16>(l, lane, &cidx, Add{});
            if ((lane & (32 / C - 1)) == 0) rd[warp][cidx] = sum;
            const bool w_ok = wait(&obar[tl & 1], (uint32_t)((tl >> 1) & 1));
            tc::fence_after_sync();
            if (!w_ok) give_up();
            if (group_or(1, kSoft, !w_ok || *reinterpret_cast<volatile int*>(&s_fail) != 0)) {
                failed = true;
                return;
            }
            const bool last = whole;
            if (tid < C) {  // (a thread a column: the same in every thread is many instructions)
                const float L = (rd[0][tid] + rd[1][tid]) + (rd[2][tid] + rd[3][tid]);
                const int n = done.n + tid / H;
                float f = L == 0.0f ? 0.0f : 1.0f / L;
                if (last && p.gate != nullptr && L != 0.0f && n < p.N) f = gated(p, (int64_t)n * p.Hq + (int64_t)done.g * H + tid % H, f);
                s_factor[tid] = f;
                if (!last) p.states[((int64_t)2 * blockIdx.x + (begins ? 1 : 0)) * S::kState + C + tid] = L;
            }
            group_or(1, kSoft, false);
            float o[C];
            {
                constexpr int n = C < 16 ? 16 : C;  // (fewer than 16 columns: both parts in one load)
                float a[n], b[n];
                const uint32_t ob = lanes + 2 * S::NS;
#pragma unroll
                for (int c = 0; c < n; c += 16) {
                    tc::ld16(ob + c, *reinterpret_cast<float(*)[16]>(a + c));
                    if (C >= 16) tc::ld16(ob + C + c, *reinterpret_cast<float(*)[16]>(b + c));
                }
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = a[c] + (C >= 16 ? b[c] : a[(C + c) % n]);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float f = s_factor[c];
                o[c] = f == 0.0f ? 0.0f : o[c] * f;
            }
            if constexpr (R > 1) {  // values that were cleared, in the rows that see them
                const int2 cl = s_cleared[(segs - 1) & 1];
                if (__builtin_expect(cl.x <= cl.y, 0)) {
                    const unsigned long long runs = s_runs[(segs - 1) & 1];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (done_set.b[r] < 0) continue;
                        const int from = max(cl.x, p.window > 0 ? max(0, done_set.pos[r] - p.window + 1) : 0);
                        const float v = not_finite(p, done_set.b[r], done.g, key, from, min(cl.y, done_set.pos[r]), runs);
                        if (v != 0.0f)
#pragma unroll
                            for (int h = 0; h < H; ++h)
                                if (s_factor[r * H + h] != 0.0f) o[r * H + h] += v;
                    }
                }
            }
            if (last) {
                uint16_t* to = p.out + ((int64_t)done.n * p.Hq + (int64_t)done.g * H) * 128 + key;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (R > 1 && done_set.b[c / H] == -1) continue;
                    to[((int64_t)(c / H) * p.Hq + c % H) * 128] = f32_to_bf16_bits(o[c]);
                }
            } else {  // CTAs first .. last share the item; each leaves its state, which the join kernel reads
                float* st = p.states + ((int64_t)2 * blockIdx.x + (begins ? 1 : 0)) * S::kState;
#pragma unroll
                for (int c = 0; c < C; ++c) st[2 * C + c * 128 + key] = o[c];
                if (key == 0)
#pragma unroll
                    for (int c = 0; c < C; ++c) st[c] = -(c & 1 ? neg_m[c / 2].y : neg_m[c / 2].x);
            }
            if (!whole && begins && tid == 0) {
                if (few)
                    p.shared_items[item0] = make_int4(done.n, done.g, rs.first, rs.last);
                else
                    p.shared_items[blockIdx.x] = make_int4(done.n, done.g, (int)blockIdx.x, (int)((done_begin + done.tiles - 1) / per));
            }
        };

        int nitem = item0, off = off0;
        for (int left = run;;) {
            if (left > 0) {
                it = rs.it;
                if (t > 0) {
                    it.tiles = 0;
                    while (nitem < items && (it = item_of<PICKS, R>(p, nitem)).tiles <= off) ++nitem;
                }
                if (nitem >= items) {
                    give_up();
                    break;
                }
                ++nitem;
                if constexpr (R > 1) set = rows_at<R>(p, it.n);
                build_q();
            }
            if (t > 0) epilogue();
            if (failed || left <= 0) break;
            if (tid == 0) {
                if (R == 1 && it.b == -2) raise_status(p.status, kDevRange);
                if constexpr (R > 1) {
                    s_cleared[segs & 1] = make_int2(INT32_MAX, -1);  // (taken by segment segs - 2, which is through)
                    s_runs[segs & 1] = 0;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (set.b[r] == -2) raise_status(p.status, kDevRange);
                }
                if (PICKS && it.b >= 0) {
                    const int n = p.sel_count[(int64_t)it.n * p.G + it.g];
                    if (n < 0 || n > p.top_k) raise_status(p.status, kDevRange);
                }
            }
            const int seg = min(it.tiles - off, left);
            done = it;
            done_set = set;
            ++segs;
            done_begin = start + (run - left) - off;
            whole = seg == it.tiles;
            begins = off == 0;
            left -= seg;
            off = 0;
#pragma unroll
            for (int c = 0; c < C / 2; ++c) {
                neg_m[c] = both(kNone);
                l_part[c] = both(0.0f);
            }
            for (int i = 0; i < seg; ++i, ++t) {
                // (tile t - 2's second product is done too: the first product of this one waited for it)
                bool w_ok = wait(&sbar[t & 1], (uint32_t)((t >> 1) & 1));
                tc::fence_after_sync();
                const uint32_t me = ring[t & (kRing - 1)][q];
                uint32_t seen = me >> (key & 7) & 1u;  // the item's rows that see the key
                if constexpr (R > 1) {
                    const int tok = s_t0[t & (kRing - 1)] + key;
                    const uint32_t rows = (uint32_t)s_note[t & (kRing - 1)] >> kRowsShift;
                    seen = 0;
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if ((me & 256u) && (rows >> r & 1u) && tok <= set.pos[r] && (p.window == 0 || tok > set.pos[r] - p.window)) seen |= 1u << r;
                }
                auto sees = [&](int c) { return (seen >> (c / H) & 1u) != 0; };
                // s[c] = q . k in log2 units, y[c] that less the running maximum
                float2 s[C / 2], y[C / 2];
#pragma unroll
                for (int c0 = 0; c0 < C; c0 += 16) {
                    float x[16];
                    tc::ld16(lanes + (uint32_t)(S::NS * (t & 1) + c0), x);
#pragma unroll
                    for (int c = 0; c < 16 && c < C; c += 2) s[(c0 + c) / 2] = mul2(make_float2(x[c], x[c + 1]), both(p.scale_log2));
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    y[c / 2] = add2(s[c / 2], neg_m[c / 2]);
                    if (sees(c)) top = fmaxf(top, fmaxf(y[c / 2].x, y[c / 2].y));
                }
                // The running maxima move when a key passes one by more than the slack; l and O are rescaled
                // then.  Every softmax thread takes the same steps.
                if (!w_ok) give_up();
                if (__builtin_expect(group_or(1, kSoft, top > kSlack || !w_ok), 0)) {
                    if (*reinterpret_cast<volatile int*>(&s_fail) != 0) failed = true;
                    float alpha[C];
                    int cidx = 0;
#pragma unroll
                    for (int c = 0; c < C; ++c) alpha[c] = sees(c) ? (c & 1 ? s[c / 2].y : s[c / 2].x) : -INFINITY;
                    const float wmax = fold<C, 16>(alpha, lane, &cidx, Max{});
                    float(&rd)[4][C] = red[t & 1];
                    if ((lane & (32 / C - 1)) == 0) rd[warp][cidx] = wmax;
                    if (group_or(1, kSoft, failed)) {
                        failed = true;
                        break;
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float tmax = fmaxf(fmaxf(rd[0][c], rd[1][c]), fmaxf(rd[2][c], rd[3][c]));
                        float& neg = c & 1 ? neg_m[c / 2].y : neg_m[c / 2].x;
                        float& l = c & 1 ? l_part[c / 2].y : l_part[c / 2].x;
                        const bool moves = tmax > kSlack - neg || (neg == kNone && tmax > -INFINITY);
                        const float a = ex2(-neg - tmax);
                        alpha[c] = moves ? a : 1.0f;
                        neg = moves ? -tmax : neg;
                        l *= alpha[c];
                    }
#pragma unroll
                    for (int c = 0; c < C; c += 2) y[c / 2] = add2(s[c / 2], neg_m[c / 2]);
                    if (i > 0) {
                        w_ok = wait(&obar[(t - 1) & 1], (uint32_t)(((t - 1) >> 1) & 1));
                        tc::fence_after_sync();
#pragma unroll
                        for (int c = 0; c < S::NO; c += 16) {
                            float o[16];
                            tc::ld16(lanes + 2 * S::NS + c, o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] *= alpha[(c + x) % C];
                            tc::st16(lanes + 2 * S::NS + c, o);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, seen != (1u << R) - 1u)) {  // (what is not seen may have anything for a score)
#pragma unroll
                    for (int c = 0; c < C; c += 2) y[c / 2] = sees(c) ? y[c / 2] : both(-INFINITY);
                }
                // A weight in two bf16 parts: its first 8 bits, and the next 8.  The second is above zero where the weight
                // is (its last bit is set), so that an infinite value meets two positive numbers.
                uint32_t hi[C / 2], lo[C / 2];
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    const float2 w = make_float2(ex2(y[c / 2].x), ex2(y[c / 2].y));
                    l_part[c / 2] = add2(l_part[c / 2], w);
                    const uint32_t a = __float_as_uint(w.x), b = __float_as_uint(w.y);
                    hi[c / 2] = __byte_perm(a, b, 0x7632);
                    lo[c / 2] = pack_bf16x2(__uint_as_float(a | 1u) - __uint_as_float(a & 0xffff0000u),
                                            __uint_as_float(b | 1u) - __uint_as_float(b & 0xffff0000u));
                }
                uint8_t* pb = pt + (t & 1) * S::kPBytes + q * S::kPGroup + (key & 7) * 16;
                if constexpr (C == 4) {
                    *reinterpret_cast<uint4*>(pb) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                } else {
#pragma unroll
                    for (int x = 0; x < C / 8; ++x) {
                        *reinterpret_cast<uint4*>(pb + x * 128) = make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
                        *reinterpret_cast<uint4*>(pb + (C / 8 + x) * 128) =
                            make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
                    }
                }
                // A copied V row that no row of the item sees is zeroed: the cache may hold anything there, and a zero
                // weight must meet a finite value.  Where some rows see it and others do not, what is not finite is, and the
                // token noted for the rows that see it.
                const uint32_t with = R == 1 ? 1u : rows_with_keys(set);
                if (__builtin_expect((me & 256u) && (seen & with) != with, 0)) {
                    const int slot = (t + 1 < run ? 2 * t + 2 : 2 * t + 1) % S::kSlots;
                    w_ok &= wait(&vfull[t & 3], (uint32_t)((t >> 2) & 1));
                    uint4* vr = reinterpret_cast<uint4*>(slots + slot * kSlotBytes + q * kRegionBytes + (key & 7) * 128);
                    if (R == 1 || seen == 0) {
#pragma unroll
                        for (int x = 0; x < 8; ++x) vr[x] = vr[64 + x] = make_uint4(0, 0, 0, 0);
                    } else {
                        bool any = false;
#pragma unroll 1
                        for (int i16 = 0; i16 < 16; ++i16) {  // (lanes of a region on different banks)
                            uint4& at = vr[(i16 >> 3) * 64 + ((i16 ^ key) & 7)];
                            const uint4 x = at;
                            uint32_t xs[4] = {x.x, x.y, x.z, x.w}, bad = 0;
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const uint32_t b = ((xs[z] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // an exponent of all ones
                                xs[z] &= ~((b >> 15) * 0xffffu);
                                bad |= b;
                            }
                            if (bad) {
                                at = make_uint4(xs[0], xs[1], xs[2], xs[3]);
                                any = true;
                            }
                        }
                        if (any) {
                            const int tok = s_t0[t & (kRing - 1)] + key;
                            atomicMin(&s_cleared[(segs - 1) & 1].x, tok);
                            atomicMax(&s_cleared[(segs - 1) & 1].y, tok);
                            atomicOr(&s_runs[(segs - 1) & 1], 1ull << (tok >> 7 & 63));
                        }
                    }
                }
                fence_proxy_async();
                tc::fence_before_sync();
                if (!w_ok) give_up();  // (the warps leave together at the next barrier)
                __syncwarp();
                if (lane == 0) arrive(&pbar[t & 1]);
            }
            if (failed) break;
        }
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
        cudaError_t e1 = cudaFuncSetAttribute(paged_attn_bf16_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
        if (e1 != cudaSuccess) return e1;
        return cudaFuncSetAttribute(paged_attn_bf16_kernel<S>, cudaFuncAttributePreferredSharedMemoryCarveout,
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
    e = cudaLaunchKernelEx(&cfg, paged_attn_bf16_kernel<S>, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    const int items = (p.N + S::R - 1) / S::R * p.G;
    if (2 * items <= (int)cfg.gridDim.x) cfg.gridDim.x = (unsigned)items;  // (the entries are by item then)
    cfg.gridDim.y = S::C;
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
    if (p.sel_ids != nullptr)  // (16 heads' weights leave room for one CTA an SM)
        return launch_shape<Shape<H, 1, true, H == 16 ? 1 : 2>>(p, kmap, vmap, num_sms, stream, pdl);
    // Two or four rows of a sequence read its keys together where it has that many.  With 8 heads a group, microseconds alone and
    // together: 2 rows of each of 4 sequences of 8,192 tokens 24 and 19, of 32,768 tokens 68 and 52; 4 rows of each of 8 of
    // 8,192 61 and 41, of 32,768 314 and 98; 4 rows of one of 32,768 34 and 21.  The longer chain of a tile shows where all rows'
    // keys are few: 4 rows of one sequence of 8,192 15 and 17, of each of 4 of 1,000 11.6 and 16.3, of each of 8 of 1,000
    // 17.8 and 18.6, 2 rows of each of 16 in a window of 512 12.1 and 15.5.  (The host knows what the table can hold, not the
    // lengths.)
    const int64_t cap = (int64_t)p.pages.table_len * p.pages.page_tokens;
    const int64_t keys = (p.window > 0 && p.window < cap ? p.window : cap) * p.N * p.G;  // at most, of all rows and groups
    const bool few_keys = keys <= 1 << 17;
    if constexpr (H <= 8)
        if (!few_keys && p.N >= (int64_t)3 * p.B) return launch_shape<Shape<H, 4, false, 1>>(p, kmap, vmap, num_sms, stream, pdl);
    if (!few_keys && p.N >= (int64_t)2 * p.B) return launch_shape<Shape<H, 2, false, 1>>(p, kmap, vmap, num_sms, stream, pdl);
    // Many tiles are shared out finer by two CTAs an SM: 16 rows of 16K to 32K tokens 124 us against 134 with one, one of
    // 524,288 159 against 161, 16 of 4K to 8K with 4 heads 40 against 41; 32 rows of 512 in a window 13.7 against 11.3.
    if constexpr (H <= 8)
        if (keys >= 1 << 19) return launch_shape<Shape<H, 1, false, 2>>(p, kmap, vmap, num_sms, stream, pdl);
    return launch_shape<Shape<H, 1, false, 1>>(p, kmap, vmap, num_sms, stream, pdl);
}

}  // namespace

cudaError_t launch_paged_attention_bf16(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   int num_sms, cudaStream_t stream, bool pdl) {
    switch (p.Hq / p.G) {
        case 4: return launch_heads<4>(p, kmap, vmap, num_sms, stream, pdl);
        case 8: return launch_heads<8>(p, kmap, vmap, num_sms, stream, pdl);
        case 16: return launch_heads<16>(p, kmap, vmap, num_sms, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace step5
