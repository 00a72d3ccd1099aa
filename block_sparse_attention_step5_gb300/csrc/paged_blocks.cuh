// paged_blocks.cuh -- what the kernels share that attend blocks of rows of a paged cache together: the tiles of keys
// of a block's rows, their split over the CTAs, the stores of head rows, and the joins of the items that CTAs share.
#pragma once

#include "paged_device.cuh"

namespace step5 {

namespace {

constexpr int kTile = 16;                       // regions of a tile of keys
constexpr int kStateFloats = 256 * 130;         // of a partial state: (m, l) of each head row, o as [16][256 head rows][8 dims]

template <int HQ_>
struct Shape {
    static constexpr int HQ = HQ_;
    static constexpr int RB = 128 / HQ;         // rows of a row tile
    static constexpr int NB = 2 * RB;           // rows of a block
    static constexpr int RL = (NB + 31) / 32;   // rows of a lane in a walk
};

struct Row {
    int b, pos, lo;  // keys: tokens lo .. pos of sequence b; b = -1: padding or past N, -2: out of range (zeros)
};

__device__ __forceinline__ Row row_of(const PagedAttnParams& p, int b, int pos) {
    Row r{b, pos, 0};
    if (r.b == -1) return r;
    if (r.b < 0 || r.b >= p.B || r.pos < 0 || r.pos >= p.pages.page_tokens * p.pages.table_len) {  // (fits int32)
        r.b = -2;
        return r;
    }
    r.lo = p.window > 0 ? max(0, r.pos - p.window + 1) : 0;
    return r;
}
__device__ __forceinline__ Row row_at(const PagedAttnParams& p, int n) {
    return n < p.N ? row_of(p, p.row_seq[n], p.row_pos[n]) : Row{-1, -1, 0};
}

// The tiles of a block of rows as a warp walks them: those of each of its sequences in turn.
template <class S>
struct Walk {
    Row mine[S::RL];     // rows lane, lane + 32 of the block
    uint64_t valid, bad; // rows with keys, rows out of range
    uint64_t todo;       // not yet walked
    int b, lo, hi, max_lo, min_hi;  // this pass: sequence, first and last token; tokens that all of its rows see
    uint64_t rows;       //   and the block's rows in it
    int r0, regions, tiles, at;     // first region, regions, tiles, tile in the pass

    __device__ __forceinline__ uint64_t votes(bool (*f)(const Row&, int), int arg) const {
        uint64_t v = 0;
#pragma unroll
        for (int i = 0; i < S::RL; ++i) v |= (uint64_t)__ballot_sync(0xffffffffu, f(mine[i], arg)) << (32 * i);
        return v;
    }
    // Asks for a block's rows; what open() then takes.
    struct Rows {
        int seq[S::RL], pos[S::RL];
    };
    static __device__ __forceinline__ Rows fetch(const PagedAttnParams& p, int n0, int lane) {
        Rows r;
#pragma unroll
        for (int i = 0; i < S::RL; ++i) {
            const int n = n0 + lane + 32 * i;
            const bool in = lane + 32 * i < S::NB && n < p.N;
            r.seq[i] = in ? p.row_seq[n] : -1;
            r.pos[i] = in ? p.row_pos[n] : -1;
        }
        return r;
    }
    // At the first tile of these rows; returns how many there are.
    __device__ __forceinline__ int open(const PagedAttnParams& p, const Rows& r) {
#pragma unroll
        for (int i = 0; i < S::RL; ++i) mine[i] = row_of(p, r.seq[i], r.pos[i]);
        valid = votes([](const Row& r, int) { return r.b >= 0; }, 0);
        bad = votes([](const Row& r, int) { return r.b == -2; }, 0);
        todo = valid;
        if (valid == 0) {  // one empty tile if anything is to be written
            b = -1, lo = 0, hi = -1, max_lo = 0, min_hi = -1, rows = 0, r0 = regions = at = 0;
            return tiles = bad ? 1 : 0;
        }
        pass(p);
        int t = tiles;
        if (todo) {  // several sequences: count them all, then back to the first
            while (todo) {
                pass(p);
                t += tiles;
            }
            todo = valid;
            pass(p);
        }
        return t;
    }
    __device__ __forceinline__ void pass(const PagedAttnParams& p) {
        const int lead = __ffsll((long long)todo) - 1;
        b = __shfl_sync(0xffffffffu, mine[0].b, lead & 31);
        if (S::RL > 1 && lead >= 32) b = __shfl_sync(0xffffffffu, mine[S::RL - 1].b, lead & 31);
        rows = votes([](const Row& r, int x) { return r.b == x; }, b);
        todo &= ~rows;
        int l = INT32_MAX, h = 0, ml = 0, mh = INT32_MAX;
#pragma unroll
        for (int i = 0; i < S::RL; ++i)
            if (mine[i].b == b) {
                l = min(l, mine[i].lo), h = max(h, mine[i].pos);
                ml = max(ml, mine[i].lo), mh = min(mh, mine[i].pos);
            }
        lo = __reduce_min_sync(0xffffffffu, l);
        hi = __reduce_max_sync(0xffffffffu, h);
        max_lo = __reduce_max_sync(0xffffffffu, ml);
        min_hi = __reduce_min_sync(0xffffffffu, mh);
        r0 = (lo >> 3) & ~(p.box_regions - 1);
        regions = (hi >> 3) - r0 + 1;
        tiles = (regions + kTile - 1) / kTile;
        at = 0;
    }
    // Whether some row of the pass sees a token of region r (of each lane its own): rows that lie apart leave gaps
    // between their windows.
    __device__ __forceinline__ bool sees(int r) const {
        if (max_lo <= min_hi + 1) return r >= (lo >> 3) && r <= (hi >> 3);  // no gap: the rows' keys touch
        bool any = false;
        for (uint64_t m = rows; m; m &= m - 1) {
            const int i = __ffsll((long long)m) - 1;
            int l = __shfl_sync(0xffffffffu, mine[0].lo, i & 31), h = __shfl_sync(0xffffffffu, mine[0].pos, i & 31);
            if (S::RL > 1 && i >= 32) {
                l = __shfl_sync(0xffffffffu, mine[S::RL - 1].lo, i & 31);
                h = __shfl_sync(0xffffffffu, mine[S::RL - 1].pos, i & 31);
            }
            any = any || (r >= (l >> 3) && r <= (h >> 3));
        }
        return any;
    }
    __device__ __forceinline__ void skip(const PagedAttnParams& p, int n) {  // to n tiles further on
        while (n >= tiles - at && todo) {
            n -= tiles - at;
            pass(p);
        }
        at += n;
    }
};

// A CTA's run of tiles: those from `start` on, of the tiles of all items (blocks of rows, group after group).
struct BlockRun {
    int64_t of_group, total, per, start;  // tiles of a group, of all, of a run
    int run, g0;                          // the run's tiles and first group
    bool dealt;                           // back to front: item dealt_item(round) of each round instead
};
// The item (block, group) of a CTA in a round of items dealt out back to front; false past the last.
template <class S>
__device__ __forceinline__ bool dealt_item(const PagedAttnParams& p, int round, int& blk, int& g) {
    const int blocks = (p.N + S::NB - 1) / S::NB, c = (int)blockIdx.x, n = (int)gridDim.x;
    const int k = round * n + (round & 1 ? n - 1 - c : c);
    blk = blocks - 1 - k / p.G;
    g = k % p.G;
    return k < blocks * p.G;
}
template <int THREADS>
struct BlockRunSmem {
    int64_t scan[THREADS / 32];
    int blk, off;  // the run's first block, and tile in it
};

// The blocks' tiles (the same for every group), a warp to a block, then this CTA's run of the tiles of all groups
// (every thread calls it, and the block meets at a barrier behind it).  tiles: room for a number a block.
// WHOLE > 0: whole items go to a CTA instead where that takes the busiest one at most WHOLE tiles more than an equal
// share (an item counting its tiles and ITEM more), dealt out in the items' order (an item goes by its middle tile) or from the last block back to the first, every other
// round in the CTAs' reverse order (a chunk's last blocks have the most keys, so that large ones meet small ones),
// whichever is better; tiles then has room for 4 kChunkMaxCtas numbers more.
template <class S, int THREADS, int WHOLE = 0, int ITEM = 0>
__device__ __forceinline__ BlockRun take_run(const PagedAttnParams& p, BlockRunSmem<THREADS>& s, int* tiles) {
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int blocks = (p.N + S::NB - 1) / S::NB;
    BlockRun r;
    auto ahead = Walk<S>::fetch(p, warp * S::NB, lane);
    for (int i = warp; i < blocks; i += THREADS / 32) {
        const auto rows = ahead;
        ahead = Walk<S>::fetch(p, (i + THREADS / 32) * S::NB, lane);
        Walk<S> w;
        const int t = w.open(p, rows);
        if (lane == 0) tiles[i] = t;
    }
    __syncthreads();
    const int chunk = (blocks + THREADS - 1) / THREADS, i0 = min(blocks, tid * chunk), i1 = min(blocks, i0 + chunk);
    int64_t sum = 0;
    for (int i = i0; i < i1; ++i) sum += tiles[i];
    int64_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) s.scan[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
    r.of_group = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += s.scan[w];
        r.of_group += s.scan[w];
    }
    r.total = r.of_group * p.G;
    r.per = (r.total + gridDim.x - 1) / gridDim.x;
    r.start = blockIdx.x * r.per;
    r.dealt = false;
    if constexpr (WHOLE > 0) {
        if (blocks * p.G <= 8 * kChunkMaxCtas && r.total < (1 << 24)) {  // (many items: the joins weigh little)
            // [0], [1]: tiles and costs in order; [2], [3]: dealt out.  An item costs its tiles and ITEM more.
            int(*load)[kChunkMaxCtas] = reinterpret_cast<int(*)[kChunkMaxCtas]>(tiles + blocks);
            for (int i = tid; i < 4 * kChunkMaxCtas; i += THREADS) load[0][i] = 0;
            if (tid == 0) s.blk = INT32_MAX;
            __syncthreads();
            const int n = (int)gridDim.x, of_group = (int)r.of_group + ITEM * blocks, per = (of_group * p.G + n - 1) / n;
            for (int g = 0; g < p.G; ++g) {
                int at = g * of_group + (int)before + ITEM * i0;
                for (int i = i0; i < i1; at += tiles[i] + ITEM, ++i)
                    if (tiles[i] > 0) {
                        const int cost = tiles[i] + ITEM, cta = (2 * at + cost) / (2 * per);
                        const int k = (blocks - 1 - i) * p.G + g, in = k % n, to = k / n & 1 ? n - 1 - in : in;
                        atomicAdd(&load[0][cta], tiles[i]);
                        atomicAdd(&load[1][cta], cost);
                        atomicAdd(&load[2][to], tiles[i]);
                        atomicAdd(&load[3][to], cost);
                        if (cta == (int)blockIdx.x) atomicMin(&s.blk, g * blocks + i);
                    }
            }
            __syncthreads();
            int most = 0, dealt = 0;
            for (int i = lane; i < n; i += 32) most = max(most, load[1][i]), dealt = max(dealt, load[3][i]);
            most = __reduce_max_sync(0xffffffffu, most);
            dealt = __reduce_max_sync(0xffffffffu, dealt);
            if (min(most, dealt) <= per + WHOLE) {
                const int first = s.blk;
                r.dealt = dealt < most;
                r.run = load[r.dealt ? 2 : 0][blockIdx.x];
                r.g0 = r.run && !r.dealt ? first / blocks : 0;
                __syncthreads();  // (first is read)
                if (tid == 0) s.blk = first % blocks, s.off = 0;
                return r;
            }
            __syncthreads();
        }
    }
    r.run = (int)(r.start < r.total ? min(r.per, r.total - r.start) : 0);
    r.g0 = r.run ? (int)(r.start / r.of_group) : 0;
    if (r.start < r.total) {
        const int64_t in = r.start % r.of_group;
        if (in >= before && in < before + sum) {
            int64_t at = before;
            for (int i = i0; i < i1; ++i) {
                if (in < at + tiles[i]) {
                    s.blk = i;
                    s.off = (int)(in - at);
                    break;
                }
                at += tiles[i];
            }
        }
    }
    return r;
}

// Head row r (of 256) of the block from row n0: dims d0 .. d0 + 7 of its output, gated (where it has keys) and rounded.
template <class S>
__device__ __forceinline__ void write_out8(const PagedAttnParams& p, int n0, int g, int r, int d0, bool keys, const float (&v)[8]) {
    const int n = n0 + r / S::HQ;
    const int64_t at = (int64_t)n * p.Hq + (int64_t)g * S::HQ + r % S::HQ;
    float f = 1.0f;
    if (p.gate != nullptr && keys) f = 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[at])));
    *reinterpret_cast<uint4*>(p.out + at * 128 + d0) =
        make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f), pack_bf16x2(v[4] * f, v[5] * f),
                   pack_bf16x2(v[6] * f, v[7] * f));
}

// 32 bytes, in one store (a whole sector) where the buffer allows it; 16-byte aligned.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
    if (reinterpret_cast<uintptr_t>(to) & 31) {
        static_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Joins the items that CTAs of the launch before shared: a block per (CTA in which such an item begins, 16 of its
// head rows), 16 threads of 8 dims to a head row (a warp: 8 rows, 4 threads each), states in the CTAs' order.
template <class S>
__global__ void __launch_bounds__(256) join_chunk_kernel(PagedAttnParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int first = blockIdx.x, hr = blockIdx.y * 16 + (threadIdx.x >> 7) * 8 + (threadIdx.x & 7), d8 = (threadIdx.x >> 3) & 15;
    const int4 item = p.shared_items[first];
    const int last = item.w, n = item.x + hr / S::HQ;
    if (last < 0 || n >= p.N || p.row_seq[n] == -1) return;
    auto state = [&](int cta) { return p.states + ((int64_t)2 * cta + (cta == first ? 1 : 0)) * kStateFloats; };
    float M = -INFINITY;
#pragma unroll 4
    for (int i = first; i <= last; ++i) {
        const float2 ml = *reinterpret_cast<const float2*>(state(i) + 2 * hr);
        if (ml.y != 0.0f) M = fmaxf(M, ml.x);
    }
    float w = 0.0f, o[8] = {};
#pragma unroll 4
    for (int i = first; i <= last; ++i) {
        const float2 ml = *reinterpret_cast<const float2*>(state(i) + 2 * hr);
        const float4* v = reinterpret_cast<const float4*>(state(i) + 512 + d8 * 2048 + hr * 8);
        const float4 a = v[0], b = v[1];
        const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - M) * ml.y;
        w += f;
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d] = fmaf(f, x[d], o[d]);
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d] = w == 0.0f ? 0.0f : o[d] / w;
    write_out8<S>(p, item.x, item.y, hr, d8 * 8, w != 0.0f, o);
}

// The same for few items, each shared by many CTAs (one sequence's 16 rows behind 8,192 tokens: 39 CTAs an
// item, 32 us in all against 40).  First the states' weights, 32 threads to a row; then two groups of 256
// threads take every other state each, eight of them asked for at a time.
template <class S>
__global__ void __launch_bounds__(512) join_wide_kernel(PagedAttnParams p) {
    constexpr int kMore = kChunkMaxCtas / 32;
    __shared__ float sw[kChunkMaxCtas][16], part[32][16], so[256][8];
    pdl_wait();
    pdl_launch_dependents();
    const int first = blockIdx.x, tid = threadIdx.x;
    const int4 item = p.shared_items[first];
    if (item.w < 0) return;
    const int n = item.w - first + 1;
    auto state = [&](int i) { return p.states + ((int64_t)2 * (first + i) + (i == 0 ? 1 : 0)) * kStateFloats; };
    {
        const int row = tid & 15, hr = blockIdx.y * 16 + row, i0 = tid >> 4;
        float2 ml[kMore];
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < kMore; ++x) {
            ml[x] = i0 + 32 * x < n ? *reinterpret_cast<const float2*>(state(i0 + 32 * x) + 2 * hr) : make_float2(0.0f, 0.0f);
            if (ml[x].y != 0.0f) M = fmaxf(M, ml[x].x);
        }
        part[i0][row] = M;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 32; ++x) M = fmaxf(M, part[x][row]);
#pragma unroll
        for (int x = 0; x < kMore; ++x)
            if (i0 + 32 * x < n) sw[i0 + 32 * x][row] = ml[x].y == 0.0f ? 0.0f : ex2(ml[x].x - M) * ml[x].y;
        __syncthreads();
    }
    const int grp = tid >> 8, at = tid & 255, row = (at >> 7) * 8 + (at & 7), d8 = (at >> 3) & 15, hr = blockIdx.y * 16 + row;
    float w = 0.0f, o[8] = {};
#pragma unroll 8
    for (int i = grp; i < n; i += 2) {
        const float4* v = reinterpret_cast<const float4*>(state(i) + 512 + d8 * 2048 + hr * 8);
        const float4 a = v[0], b = v[1];
        const float f = sw[i][row], x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        w += f;
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d] = fmaf(f, x[d], o[d]);
    }
    if (grp == 1) {
#pragma unroll
        for (int d = 0; d < 8; ++d) so[at][d] = o[d];
        if (d8 == 0) part[0][row] = w;
    }
    __syncthreads();
    const int r = item.x + hr / S::HQ;
    if (grp == 1 || r >= p.N || p.row_seq[r] == -1) return;
    w += part[0][row];
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d] = w == 0.0f ? 0.0f : (o[d] + so[at][d]) / w;
    write_out8<S>(p, item.x, item.y, hr, d8 * 8, w != 0.0f, o);
}

// Launches the join behind a launch of cfg.
template <class S>
cudaError_t launch_join(const PagedAttnParams& p, int num_sms, cudaLaunchConfig_t cfg) {
    cfg.gridDim.y = 256 / 16;
    cfg.dynamicSmemBytes = 0;
    // at least 8 CTAs an item on average, or fewer (2,048 rows on 2K: 138 us against 152 with the wide one)
    if ((int64_t)((p.N + S::NB - 1) / S::NB) * p.G * 8 <= num_sms) {
        cfg.blockDim = dim3(512);
        return cudaLaunchKernelEx(&cfg, join_wide_kernel<S>, p);
    }
    cfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&cfg, join_chunk_kernel<S>, p);
}

}  // namespace

}  // namespace step5
