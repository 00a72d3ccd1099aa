// paged_items.cuh -- what the kernels share that attend rows of a paged cache on their own: items (a row's keys in
// a group, in tiles), their split over the CTAs, and the join of the items that CTAs share.
#pragma once

#include <type_traits>

#include "paged_device.cuh"

namespace step5 {

namespace {

constexpr int kTile = 16;            // regions of a tile

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

// Items of R rows: the keys of rows n .. n + R - 1 in group g, those of each of their sequences in turn.
template <int R>
struct RowSet {
    int b[R], pos[R];  // as the call has them; b = -1: padding or past N, -2: out of range
};
template <int R>
__device__ __forceinline__ RowSet<R> rows_at(const PagedAttnParams& p, int n) {
    RowSet<R> s;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        s.b[r] = n + r < p.N ? p.row_seq[n + r] : -1;
        s.pos[r] = n + r < p.N ? p.row_pos[n + r] : -1;
        if (s.b[r] != -1 && (s.b[r] < 0 || s.b[r] >= p.B || s.pos[r] < 0 || s.pos[r] >= p.pages.page_tokens * p.pages.table_len))
            s.b[r] = -2;
    }
    return s;
}
// One of an item's sequences: its rows (a mask) and their first and last token.
struct Pass {
    int b, lo, hi, r0, entries, tiles;
    uint32_t rows;
};
// The sequence of the first of the rows `todo`, which loses its rows.
template <int R>
__device__ __forceinline__ Pass next_pass(const PagedAttnParams& p, const RowSet<R>& s, uint32_t& todo) {
    Pass a{-1, INT32_MAX, -1, 0, 0, 0, 0u};
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
        if (todo >> r & 1u) a.b = s.b[r];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if ((todo >> r & 1u) && s.b[r] == a.b) {
            a.rows |= 1u << r;
            a.lo = min(a.lo, p.window > 0 ? max(0, s.pos[r] - p.window + 1) : 0);
            a.hi = max(a.hi, s.pos[r]);
        }
    todo &= ~a.rows;
    a.r0 = (a.lo >> 3) & ~(p.box_regions - 1);
    a.entries = (a.hi >> 3) - a.r0 + 1;
    a.tiles = (a.entries + kTile - 1) / kTile;
    return a;
}
template <int R>
__device__ __forceinline__ uint32_t rows_with_keys(const RowSet<R>& s) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) m |= s.b[r] >= 0 ? 1u << r : 0u;
    return m;
}

// Item i of R rows (of one: as above).  b: -1 without tiles, -2 with one empty tile (rows out of range alone), else 0.
template <bool PICKS, int R>
__device__ __forceinline__ Item item_of(const PagedAttnParams& p, int i) {
    if constexpr (R == 1) {
        return item_at<PICKS>(p, i);
    } else {
        const int blocks = (p.N + R - 1) / R;
        Item it{};
        it.g = i / blocks;
        it.n = (i - it.g * blocks) * R;
        const RowSet<R> s = rows_at<R>(p, it.n);
        uint32_t todo = rows_with_keys(s);
        while (todo) it.tiles += next_pass<R>(p, s, todo).tiles;
        if (it.tiles == 0) {
            it.b = -1;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (s.b[r] == -2) it.b = -2, it.tiles = 1;
        }
        return it;
    }
}

// The output v of a (row, head), number `at` of them, through its gate.
__device__ __forceinline__ float gated(const PagedAttnParams& p, int64_t at, float v) {
    return v * (1.0f / (1.0f + expf(-bf16_to_f32(p.gate[at]))));
}

// A CTA's run of tiles in shared memory: from tile `off` of item `item`; with few items the CTAs that share it.
template <int THREADS>
struct RunSmem {
    int64_t scan[THREADS / 32];
    int tiles[THREADS], item, off, run, first, last;
    Item it;  // item `item`
    uint32_t ctas[THREADS / 32][32];
};

// Splits the items' tiles over the CTAs (every thread calls it, and the block meets at a barrier behind it).  Returns
// whether there are few; of many, start is the run's first tile among all and per the tiles of a run.
template <bool PICKS, int THREADS, int R = 1>
__device__ __forceinline__ bool take_run(const PagedAttnParams& p, RunSmem<THREADS>& s, int64_t& start, int64_t& per) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, items = (p.N + R - 1) / R * p.G;
    start = 0, per = 1;
    const bool few = 2 * items <= (int)gridDim.x;
    if (few) {
        // Few items: each is cut into equal parts, one CTA a part, of at most L tiles for the
        // smallest L of 32 tried that needs no more CTAs than there are (2 L0 always does).  No CTA
        // then has parts of two items. (fewer than 2^8 items of at most 2^24 tiles a row)
        Item own{};
        if (tid < items) own = item_of<PICKS, R>(p, tid);
        const uint32_t mine = (uint32_t)own.tiles;
        s.tiles[tid] = own.tiles;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) s.scan[warp] = sum;
        if (tid == 0) s.run = 0;
        __syncthreads();
        std::conditional_t<R == 1, uint32_t, uint64_t> total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) total += (uint32_t)s.scan[w];
        const uint32_t least = max(1u, (uint32_t)(total / gridDim.x) + (total % gridDim.x ? 1u : 0u));
        uint32_t most = least + (least * (uint32_t)lane + 30u) / 31u;  // this lane's L
        uint32_t ctas = 0;
        for (int i = warp; i < items; i += THREADS / 32) ctas += ((uint32_t)s.tiles[i] + most - 1u) / most;
        s.ctas[warp][lane] = ctas;
        __syncthreads();
        ctas = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) ctas += s.ctas[w][lane];
        most = __shfl_sync(0xffffffffu, most, __ffs(__ballot_sync(0xffffffffu, ctas <= gridDim.x)) - 1);
        const int parts = (int)((mine + most - 1u) / most);
        int inc = parts;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) s.scan[warp] = inc;
        __syncthreads();
        int first = inc - parts;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w)
            if (w < warp) first += (int)s.scan[w];
        const int part = (int)blockIdx.x - first;
        if (part >= 0 && part < parts) {
            s.item = tid;
            s.it = own;
            const uint32_t each = mine / (uint32_t)parts, more = mine % (uint32_t)parts;  // (the first ones take one more)
            s.off = (int)((uint32_t)part * each + min((uint32_t)part, more));
            s.run = (int)(each + ((uint32_t)part < more ? 1u : 0u));
            s.first = first;
            s.last = first + parts - 1;
            if (part == 0) p.shared_items[tid] = make_int4(0, 0, 0, -1);  // (again below if it has several parts)
        }
        if (blockIdx.x == 0 && tid < items && mine == 0) p.shared_items[tid] = make_int4(0, 0, 0, -1);
    } else {
        // Many: the items' tiles are laid end to end and every CTA takes an equal run of them.
        if (tid == 0) {
            p.shared_items[blockIdx.x] = make_int4(0, 0, 0, -1);  // (again below if an item that other CTAs share begins here)
            s.run = 0;
        }
        const int chunk = (items + THREADS - 1) / THREADS;
        const int i0 = min(items, tid * chunk), i1 = min(items, i0 + chunk);
        int64_t sum = 0;
        for (int i = i0; i < i1; ++i) sum += item_of<PICKS, R>(p, i).tiles;
        int64_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) s.scan[warp] = inc;
        __syncthreads();
        int64_t before = inc - sum, total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += s.scan[w];
            total += s.scan[w];
        }
        per = (total + gridDim.x - 1) / gridDim.x;
        start = blockIdx.x * per;
        if (start >= before && start < before + sum) {
            int64_t at = before;
            for (int i = i0; i < i1; ++i) {
                const Item it = item_of<PICKS, R>(p, i);
                const int t = it.tiles;
                if (start < at + t) {
                    s.item = i;
                    s.it = it;
                    s.off = (int)(start - at);
                    s.run = (int)min(per, total - start);
                    break;
                }
                at += t;
            }
        }
    }
    return few;
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
    // (column c: head c % H of the item's row c / H)
    if (S::C > S::H && (item.x + c / S::H >= p.N || p.row_seq[item.x + c / S::H] == -1)) return;
    auto state = [&](int i) { return p.states + ((int64_t)2 * (first + i) + (i == 0 ? 1 : 0)) * S::kState; };
    constexpr int kDeep = 8;
    float v[kDeep];
#pragma unroll
    for (int x = 0; x < kDeep; ++x) v[x] = grp + x * GROUPS < n ? state(grp + x * GROUPS)[2 * S::C + c * 128 + d] : 0.0f;
    // the states' weights 2^(m - M) l
    float M = -INFINITY;
    for (int i = tid; i < n; i += 128 * GROUPS)
        if (state(i)[S::C + c] != 0.0f) M = fmaxf(M, state(i)[c]);
#pragma unroll
    for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    if ((tid & 31) == 0) sm[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < GROUPS * 4; ++x) M = fmaxf(M, sm[x]);
    for (int i = tid; i < n; i += 128 * GROUPS) {
        const float l = state(i)[S::C + c];
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
        o = fmaf(sw[i], state(i)[2 * S::C + c * 128 + d], o);
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
        const int64_t at = (int64_t)(item.x + c / S::H) * p.Hq + (int64_t)item.y * S::H + c % S::H;
        o = w == 0.0f ? 0.0f : o / w;
        if (p.gate != nullptr && w != 0.0f) o = gated(p, at, o);
        p.out[at * 128 + d] = f32_to_bf16_bits(o);
    }
}

}  // namespace

}  // namespace step5
