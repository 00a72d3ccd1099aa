// paged_chunk_bf16.cu -- attention over the bf16 paged cache for launches whose sequences have several rows (prompt
// chunks, drafts): the rows of a sequence share its keys.
//
//   s_t = softmax_scale (q . k_t),  p = softmax(s),  out = sum_t p_t v_t
//
// A CTA takes two tiles of 128 head rows (128 / HQ consecutive rows of the call, HQ query heads each) against
// 128 keys at a time, bf16 throughout:
//
//   S [128 head rows x 128 keys]  = q . K^T   (q and K as they lie in memory, brought by TMA)
//   O [128 head rows x 128 dims] += P . V     (P from tensor memory, in the place of its S)
//
// Two softmax threads have a head row, 64 keys of a tile each: a thread takes its half row of S into registers whole, and the
// pair needs each other only when the running maximum moves.  The row tiles take turns: while one's softmax runs,
// the tensor core has the other's two products (1,024 cycles for 128 rows against 128 keys).
//
// Unseen values.  A weight of zero must meet a finite value, but a page may hold anything where a row does not look.
// Where some row of the block does not see some key of the tile (its edges, bad pages), two warps look the tile of V over, clear
// what is not finite, and note the tokens it was found at, of those that some row sees; the rows that see one of them take it up
// again at their end, from the page itself.
//
// Work.  An item is a (block of rows, group).  Where whole items share out evenly enough they go to a CTA whole; otherwise, as over
// the e4m3 pages, the tiles of all items are laid end to end, each CTA takes an equal run, and a second kernel joins the items
// that CTAs share.
//
// What it takes, with 4 KV groups of 8 heads and pages of 64 tokens (by graph replay, join included):
//   2,048 rows behind 2,048 tokens        94 us  1.03e11 flop, 1.09 PFLOP/s (57 % of measured cuBLAS)
//   2,048 rows behind 65,536 tokens    1,471 us  2.23e12 flop, 1.52 PFLOP/s (79 %); called on end 1,650 us, 1.35 PFLOP/s: the clock
//   2,048 rows, window of 512 tokens      38 us  1.7e10 flop (9 us)
//   3 prompts of 701, 2 groups of 16      41 us  1.2e10 flop (6 us)
// A tile of keys takes its two row tiles at most 3,500 cycles (65,536 tokens: 875 tiles a CTA), of which the tensor core works 2,056.
// By clock stamps in the kernel, which stretch a tile to 4,000, each row tile's chain is half softmax (330 to fetch S, 220 maximum,
// 330 the pair's barrier, 850 weights, 240 to hand P over) and half its two products and their turn; two chains are all that tensor
// memory holds.  Around the tiles: start 8 us (sharing out 4.5, first rows, pages, q, K and product 3.5); about two tiles' time for
// each item (its first maximum, the check of its edges, the turn of the products, the epilogue).
#include <type_traits>

#include "paged_blocks.cuh"

namespace step5 {

namespace {

constexpr int kMmaWarp = 0, kLoadWarp = 1, kCheckWarp = 2, kSoftWarp = 4;  // (two that check, sixteen of softmax)
constexpr int kThreads = 20 * 32;
constexpr int kRing = 8;
constexpr int kStagesK = 3, kStagesV = 2;
constexpr uint32_t kRegionBytes = 2048, kTileBytes = kTile * kRegionBytes, kQBytes = 128 * 256;
constexpr uint32_t kTilesBytes = 2 * kQBytes + (kStagesK + kStagesV) * kTileBytes;
constexpr int kRowSegs = 4;                     // segments whose rows are in shared memory
constexpr uint32_t kCols = 512;                 // S of both row tiles (P in the first half of each), O of both
constexpr uint32_t kIdescQk = tc::instr_desc(tc::kFmtBF16, false, false, 128, 128);
constexpr uint32_t kIdescPv = tc::instr_desc(tc::kFmtBF16, false, true, 128, 128);
constexpr float kSlack = 8.0f;                  // log2 units a weight may lie above the running maximum

// Tiles that the busiest CTA may have over an equal share before items are cut: what a cut costs, a partial state and its join
// for most CTAs (window of 512: 53 us cut, 44 whole; three prompts of 701 rows 56.7 and 52.1; 2,048 rows on 2K, dealt out, 112 and 97).
constexpr int kWholeTiles = 8;
constexpr int kItemTiles = 2;  // what an item takes beside its tiles: q, the turn of the products, the epilogue

// A tile as the copying warp leaves it for the others.
struct Tile {
    uint64_t rows;       // the block's rows that the tile's sequence is of
    uint32_t ok;         // regions that can be read and hold keys
    int t0;              // first token
    uint32_t note;       // kFirst ...
    int g, n0;           // group, first row of the block
    int last;            // the CTA that has the item's last tile
    int all_lo, all_hi;  // tokens that every row of the block but padding sees
};
// A segment: the tiles of an item (group, block of rows) that a CTA has.
enum : uint32_t {
    kFirst = 1,          // the segment's first tile
    kLast = 2,           // its last
    kAll = 4,            // every row of the block but padding sees every key of the tile
    kWhole = 8,          // the segment is the whole item
    kBegins = 16,        // it has the item's first tile
    kIdle = 32           // << w: row tile w has no row of the tile's sequence
};

// Tokens of a segment that some row sees and whose values are not finite and were cleared: the first and the last (none: hi < lo), and
// of which runs of 128 tokens they are (bit: the run's number modulo 64), so that what lies between need not be searched.
struct Cleared {
    int lo, hi;
    unsigned long long runs;
};

// Shared memory behind the tiles (which start on a swizzle atom's boundary: there is no static shared memory).
template <class S>
struct Control {
    uint64_t kfull[kStagesK], kempty[kStagesK], vfull[kStagesV], vempty[kStagesV], go[kStagesV], sbar[2], pbar[2], obar[2], qbar, fbar;
    BlockRunSmem<kThreads> rs;
    Tile ring[kRing];
    int rows[kRowSegs][S::NB];   // of segment i % 4: the rows' positions; -1: padding, -2: out of range
    Cleared cleared[8];          // of segment i % 8
    float part[256];             // of each head row: a maximum or sum between its two threads
    uint32_t tmem;
    int fail;
};
template <class S>
constexpr uint32_t kSmem = kTilesBytes + (uint32_t)sizeof(Control<S>);

// Bits 15 and 31: whether either of two bf16 values is not finite (an exponent of all ones).
__device__ __forceinline__ uint32_t all_ones(uint32_t u) { return ((u & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }

// Adds to 64 values of each lane's head row (bf16 at out, or fp32 in groups of 8 at state) what is not finite in their dims, from
// dim d0 on, among the noted tokens and those first .. last of its sequence b (-1: none).  The warp looks through 32 tokens at a
// time, a token a lane, for the dims with +infinity and -infinity (NaN: both).  Rarely run, and apart from the code that is.  304
// blocks of two sequences, 16,000 tokens each, 0.53 ms: with seven such values at both ends and in the middle 0.61, with one sequence
// of nothing else 8.9.
__device__ __noinline__ void add_not_finite(const PagedAttnParams& p, const Cleared& cl, int b, int g, int d0, int first, int last,
                                            uint16_t* out, float* state) {
    constexpr uint32_t kWarp = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const unsigned long long runs = cl.runs;
    uint32_t mine[4] = {};  // this lane's row: even dims and odd dims with +infinity, and those with -infinity
    for (uint32_t todo = __ballot_sync(kWarp, b >= 0); todo;) {  // the lanes' sequences in turn
        const int of = __shfl_sync(kWarp, b, __ffs(todo) - 1);
        todo &= ~__ballot_sync(kWarp, b == of);
        const uint32_t from = (uint32_t)__reduce_min_sync(kWarp, b == of ? first : INT32_MAX);
        const uint32_t to = (uint32_t)__reduce_max_sync(kWarp, b == of ? last : 0);
        for (uint32_t t0 = from & ~31u; t0 <= to; t0 += 32) {
            if (!(runs >> (t0 >> 7 & 63) & 1u)) {
                t0 |= 96;
                continue;
            }
            const uint32_t t = t0 + lane;
            const int64_t row = t >= from && t <= to ? page_row(p.pages, p.G, of, g, (int)t) : -1;
            const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.v_pages) + row * 128 + d0);
            uint32_t any = 0, has[4] = {};
            if (row >= 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) any |= all_ones(v[i].x) | all_ones(v[i].y) | all_ones(v[i].z) | all_ones(v[i].w);
            if (any) {
#pragma unroll 1
                for (int i = 0; i < 32; ++i) {
                    const uint32_t x = reinterpret_cast<const uint32_t*>(v)[i];
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const uint32_t e = x >> (16 * odd) & 0xffffu;
                        if ((e & 0x7f80u) != 0x7f80u) continue;
                        if ((e & 0x7fu) || !(e & 0x8000u)) has[odd] |= 1u << i;
                        if ((e & 0x7fu) || (e & 0x8000u)) has[2 + odd] |= 1u << i;
                    }
                }
            }
            uint32_t m = __ballot_sync(kWarp, any != 0);
            if (m == 0) continue;
            if (__all_sync(kWarp, b != of || (first <= (int)t0 && (uint32_t)last >= t0 + 31))) {  // every row sees all 32
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t all = __reduce_or_sync(kWarp, has[i]);
                    if (b == of) mine[i] |= all;
                }
            } else {
                for (; m; m &= m - 1) {
                    const int j = __ffs(m) - 1;
                    const bool sees = b == of && (uint32_t)first <= t0 + j && t0 + j <= (uint32_t)last;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t one = __shfl_sync(kWarp, has[i], j);
                        if (sees) mine[i] |= one;
                    }
                }
            }
        }
    }
#pragma unroll 1
    for (int d = 0; d < 64; ++d) {
        const bool up = mine[d & 1] >> (d >> 1) & 1u, down = mine[2 + (d & 1)] >> (d >> 1) & 1u;
        if (!up && !down) continue;
        const float x = up && down ? NAN : up ? INFINITY : -INFINITY;
        if (state != nullptr)
            state[(d >> 3) * 2048 + (d & 7)] += x;
        else
            out[d] = f32_to_bf16_bits(bf16_to_f32(out[d]) + x);
    }
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_bf16_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, PagedAttnParams p) {
    constexpr int HQ = S::HQ, RB = S::RB, NB = S::NB;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;                               // [row tile][half of the dims][128 head rows][128 B], 128-byte swizzle
    uint8_t* ks = qs + 2 * kQBytes;                   // [stage][16 regions][half][8 tokens][128 B], swizzled
    uint8_t* vs = ks + kStagesK * kTileBytes;
    Control<S>& sm = *reinterpret_cast<Control<S>*>(smem + kTilesBytes);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int blocks = (p.N + NB - 1) / NB;

    if (tid == 0) {
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        for (int i = 0; i < kStagesK; ++i) {
            mbar_init(&sm.kfull[i], 1);
            mbar_init(&sm.kempty[i], 1);
        }
        for (int i = 0; i < kStagesV; ++i) {
            mbar_init(&sm.vfull[i], 1);
            mbar_init(&sm.vempty[i], 1);
            mbar_init(&sm.go[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.sbar[i], 2);
            mbar_init(&sm.pbar[i], 8);
            mbar_init(&sm.obar[i], 2);
        }
        mbar_init(&sm.qbar, 1);
        mbar_init(&sm.fbar, 1);
        fence_mbar_init();
        sm.fail = 0;
    }
    if (tid < 8) sm.cleared[tid] = Cleared{INT32_MAX, -1, 0};
    if (warp == kMmaWarp) tc::alloc(&sm.tmem, kCols);
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) p.shared_items[blockIdx.x].w = -1;
    const BlockRun of = take_run<S, kThreads, kWholeTiles, kItemTiles>(p, sm.rs, reinterpret_cast<int*>(smem));  // (nothing is copied yet)
    const int64_t per = of.per, start = of.start;
    fence_proxy_async();  // (the copies write where the tiles' numbers were)
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem;
    const int run = of.run, blk0 = sm.rs.blk, off0 = sm.rs.off, g0 = of.g0;

    // The copying warp walks the run's segments: item (group, block), tiles off .. off + n - 1 of it.
    // next() returns false when there is none (the rows have changed under the kernel).
    struct Segment {
        int g, blk, off, n, nt;
    };
    int round = 0;
    auto next = [&](Segment& s, Walk<S>& w, int left) -> bool {
        for (;;) {
            if (of.dealt) {
                if (!dealt_item<S>(p, round++, s.blk, s.g)) return false;
            } else if (s.blk >= blocks) {
                s.blk = 0;
                if (++s.g >= p.G) return false;
            }
            s.nt = w.open(p, w.fetch(p, s.blk * NB, lane));
            if (s.nt > s.off) break;
            ++s.blk;
        }
        s.n = min(s.nt - s.off, left);
        return true;
    };
    auto give_up = [&] {
        raise_status(p.status, kDevTimeout);
        atomicExch(&sm.fail, 1);
    };
    auto failed = [&](bool ok) {  // for a whole warp
        if (!__all_sync(0xffffffffu, ok && *reinterpret_cast<volatile int*>(&sm.fail) == 0)) {
            if (lane == 0) give_up();
            return true;
        }
        return false;
    };

    if (run == 0) {
        // nothing to do
    } else if (warp == kLoadWarp) {
        // ---------------- copies: K_0, q, K_1, V_0, K_2, V_1, ..., q of a new block behind the last product of the one before;
        // lane l looks up region l % 16 of tile l / 16 of two
        constexpr uint64_t kRows0 = (1ull << RB) - 1ull;  // rows of the first row tile
        const int k = p.box_regions, q = lane & 15;
        Walk<S> w{};
        Segment s{g0, blk0, off0, 0, 0};
        int left = run, seg_left = 0, issued_k = 0, issued_v = 0, segs = 0, last = 0;
        int b_row = -1, n_row = -1, batch = -1, done = 0;
        uint32_t b_seen = 0, n_seen = 0;  // lanes whose region some row sees
        bool ok = true;
        auto look = [&](int of) {
            const int r = w.r0 + (of * 2 + (lane >> 4)) * kTile + q;
            n_row = -1;
            n_seen = __ballot_sync(0xffffffffu, w.sees(r));
            if (n_seen >> (lane & ~(k - 1)) & ((1u << k) - 1u)) {  // (some region of its box)
                n_row = (int)page_row(p.pages, p.G, w.b, s.g, r * 8);
                if (n_row < 0) raise_status(p.status, kDevRange);
            }
        };
        int row = -1;  // of the tile whose V is next
        for (int t = 0; t <= run; ++t) {
            int nrow = -1;
            bool first = false;
            if (t < run) {
                first = seg_left == 0;
                if (first) {
                    if (!next(s, w, left)) {
                        ok = false;
                        break;
                    }
                    last = (int)((start + (run - left) - s.off + s.nt - 1) / per);
                    w.skip(p, s.off);
                    seg_left = s.n;
                    left -= s.n;
                    batch = -1, done = 0;
                } else if (w.at + 1 < w.tiles) {
                    ++w.at;
                } else {
                    w.pass(p);
                    batch = -1, done = 0;
                }
                --seg_left;
                if (batch != w.at >> 1) {
                    if (!done) look(w.at >> 1);
                    batch = w.at >> 1;
                    b_row = n_row, b_seen = n_seen, done = 0;
                } else if ((batch + 1) * 2 < w.tiles) {
                    look(batch + 1);
                    done = 1;
                }
                const int from = (w.at & 1) * 16 + q;
                nrow = __shfl_sync(0xffffffffu, b_row, from);
                const uint32_t oks = __ballot_sync(0xffffffffu, nrow >= 0 && (b_seen >> from & 1u)) & 0xffffu;
                if (t >= kStagesK && !wait(&sm.kempty[t % kStagesK], (uint32_t)((t / kStagesK - 1) & 1))) ok = false;
                if (failed(ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int t0 = (w.r0 + w.at * kTile) * 8;
                    const bool all = oks == 0xffffu && w.rows == w.valid && w.bad == 0 && t0 >= w.max_lo && t0 + 127 <= w.min_hi;
                    Tile& tl = sm.ring[t & (kRing - 1)];
                    tl.rows = w.rows;
                    tl.ok = oks;
                    tl.t0 = t0;
                    tl.note = (first ? kFirst : 0u) | (seg_left == 0 ? kLast : 0u) | (all ? kAll : 0u) | (s.n == s.nt ? kWhole : 0u) |
                              (s.off == 0 ? kBegins : 0u) | ((w.rows & kRows0) == 0 ? kIdle : 0u) | ((w.rows & ~kRows0) == 0 ? kIdle << 1 : 0u);
                    tl.g = s.g;
                    tl.n0 = s.blk * NB;
                    tl.last = last;
                    const bool one = w.rows == w.valid && w.bad == 0;
                    tl.all_lo = one ? w.max_lo : INT32_MAX;
                    tl.all_hi = one ? w.min_hi : -1;
                }
                if (first)  // (the softmax is past tile t - 4, and with it past the first tile of segment i - 4)
#pragma unroll
                    for (int i = 0; i < S::RL; ++i)
                        if (lane + 32 * i < NB) sm.rows[segs & (kRowSegs - 1)][lane + 32 * i] = w.mine[i].b < 0 ? w.mine[i].b : w.mine[i].pos;
                const int n0 = s.blk * NB, g = s.g;
                if (seg_left == 0) {  // on to the next item
                    s.off = 0;
                    ++s.blk;
                }
                if (!(lane < 16 && (q & (k - 1)) == 0)) nrow = -1;
                const uint32_t have = __ballot_sync(0xffffffffu, nrow >= 0);
                __syncwarp();
                const int st = t % kStagesK;
                if (lane == 0) mbar_arrive_expect_tx(&sm.kfull[st], (uint32_t)__popc(have) * kRegionBytes * k);
                __syncwarp();
                if (nrow >= 0) tma_load_4d(ks + st * kTileBytes + q * kRegionBytes, &kmap, &sm.kfull[st], 0, 0, 0, nrow >> 3);
                issued_k = t + 1;
                if (first && t == 0 && lane == 0) {
                    mbar_arrive_expect_tx(&sm.qbar, 2 * kQBytes);
                    tma_load_4d(qs, &qmap, &sm.qbar, 0, g * HQ, n0, 0);
                    tma_load_4d(qs + kQBytes, &qmap, &sm.qbar, 0, g * HQ, n0 + RB, 0);
                }
                if (first) ++segs;
                __syncwarp();
            }
            if (t > 0) {
                const int v = t - 1, st = v % kStagesV;
                if (v >= kStagesV && !wait(&sm.vempty[st], (uint32_t)((v / kStagesV - 1) & 1))) ok = false;
                if (failed(ok)) {
                    ok = false;
                    break;
                }
                const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
                if (lane == 0) mbar_arrive_expect_tx(&sm.vfull[st], (uint32_t)__popc(have) * kRegionBytes * k);
                __syncwarp();
                if (row >= 0) tma_load_4d(vs + st * kTileBytes + q * kRegionBytes, &vmap, &sm.vfull[st], 0, 0, 0, row >> 3);
                issued_v = t;
                if (t < run && first) {  // the products of the block before have read its q
                    if (!wait(&sm.kempty[v % kStagesK], (uint32_t)((v / kStagesK) & 1))) ok = false;
                    if (failed(ok)) {
                        ok = false;
                        break;
                    }
                    const Tile& tl = sm.ring[t & (kRing - 1)];
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sm.qbar, 2 * kQBytes);
                        tma_load_4d(qs, &qmap, &sm.qbar, 0, tl.g * HQ, tl.n0, 0);
                        tma_load_4d(qs + kQBytes, &qmap, &sm.qbar, 0, tl.g * HQ, tl.n0 + RB, 0);
                    }
                    __syncwarp();
                }
            }
            row = nrow;
        }
        if (!ok && lane == 0) {  // let the copies issued land (bounded) before the shared memory goes away
            give_up();
            for (int i = max(0, issued_k - kStagesK); i < issued_k; ++i) wait(&sm.kfull[i % kStagesK], (uint32_t)((i / kStagesK) & 1));
            for (int i = max(0, issued_v - kStagesV); i < issued_v; ++i) wait(&sm.vfull[i % kStagesV], (uint32_t)((i / kStagesV) & 1));
            if (segs > 0) wait(&sm.qbar, (uint32_t)((segs - 1) & 1));
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------- products, of the row tiles in turn: P V of a tile, then Q K of the next, whose S takes P's
        // place (products of one thread run in order).  Behind a segment's last tile q changes: both
        // P V go first.  One thread does it all: it keeps the tensor core fed only if little stands between two products.
        if (elect()) {
            const uint64_t dq = tc::smem_desc(smem_u32(qs), 16, 1024, tc::kSwizzle128);
            const uint64_t dk = tc::smem_desc(smem_u32(ks), 16, kRegionBytes, tc::kSwizzle128);
            const uint64_t dv = tc::smem_desc(smem_u32(vs), 1024, kRegionBytes, tc::kSwizzle128);
            uint32_t kst = 0, vst = 0, vpar = 0, segs = 0, note = 0;
            bool ok = wait(&sm.kfull[0], 0) && wait(&sm.qbar, 0);
            uint32_t begun = 0;  // row tiles that have had a product of the segment
            // Step t: P V of tile t, Q K of tile t + 1 (from t = -1 on), of the row tiles in turn.
            for (int t = -1; t < run && ok; ++t) {
                const uint32_t of = note;
                const bool more = t + 1 < run, turn = t < 0 || (of & kLast) != 0;
                if (of & kFirst) begun = 0;
                if (t >= 0) {
                    if (!(ok = wait(&sm.go[vst], vpar))) break;  // V of this tile and K of the next are there
                    if (more && ++kst == kStagesK) kst = 0;
                }
                tc::fence_after_sync();
                if (more) note = sm.ring[(t + 1) & (kRing - 1)].note;
                const uint64_t db = dv + vst * (kTileBytes >> 4);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {  // P V 0, Q K 0, P V 1, Q K 1; at a turn both P V first
                    if (t < 0 && i < 2) continue;
                    const uint32_t w = turn ? i & 1 : i >> 1;
                    if (turn ? i < 2 : !(i & 1)) {
                        if (!(ok = wait(&sm.pbar[w], (uint32_t)(t & 1)))) break;
                        tc::fence_after_sync();
                        if (!(of & kIdle << w)) {
                            const uint32_t d = tmem + 256u + 128u * w, a = tmem + 128u * w;
#pragma unroll
                            for (int k = 0; k < 8; ++k)  // 16 keys each
                                tc::mma_f16_ts(d, a + 8u * k, db + (2 * kRegionBytes >> 4) * k, kIdescPv, (begun >> w & 1u) || k > 0);
                            begun |= 1u << w;
                        }
                        if (turn) {
                            arrive(&sm.obar[w]);  // (hands the checking warps' notes on)
                            tc::commit(&sm.obar[w]);
                        }
                        if (w == 1) tc::commit(&sm.vempty[vst]);
                    } else if (more) {
                        if (turn && w == 0 && t >= 0) {
                            if (!(ok = wait(&sm.qbar, ++segs & 1u))) break;
                            tc::fence_after_sync();
                        }
                        const uint64_t da = dq + w * (kQBytes >> 4), dk1 = dk + kst * (kTileBytes >> 4);
                        if (!(note & kIdle << w)) {
                            const uint32_t d = tmem + 128u * w;
#pragma unroll
                            for (int k = 0; k < 8; ++k)  // 16 dims each
                                tc::mma_f16(d, da + (k < 4 ? 2 * k : (kQBytes >> 5) + 2 * (k - 4)), dk1 + (k < 4 ? 2 * k : 64 + 2 * (k - 4)),
                                            kIdescQk, k > 0);
                        }
                        arrive(&sm.sbar[w]);  // (hands the tile's ring entry on, which came with its K)
                        tc::commit(&sm.sbar[w]);
                        if (w == 1) tc::commit(&sm.kempty[kst]);
                    }
                }
                if (t >= 0 && ++vst == kStagesV) vst = 0, vpar ^= 1u;
            }
            if (!ok) {  // the products issued end before their memory goes away
                give_up();
                tc::commit(&sm.fbar);
                wait(&sm.fbar, 0);
            }
        }
        __syncwarp();
    } else if (warp < kSoftWarp) {
        // ---------------- V of the tiles that not every row sees whole: what is not finite becomes zero, and is noted.  The
        // products wait for these warps alone: V of their tile, and K of the next, are there.
        const int half = warp - kCheckWarp;  // regions 8 half .. 8 half + 7
        int segs = 0;
        for (int t = 0; t < run; ++t) {
            const int st = t % kStagesV;
            if (failed(wait(&sm.vfull[st], (uint32_t)((t / kStagesV) & 1)))) break;
            const Tile& tl = sm.ring[t & (kRing - 1)];
            const uint32_t note = tl.note;
            if (note & kFirst) {
                // (segment i - 5's notes have been read: its successors' tiles have been worked on)
                if (half == 0 && lane == 0) sm.cleared[(segs + 3) & 7] = Cleared{INT32_MAX, -1, 0};
                ++segs;
            }
            if (!(note & kAll)) {
                Cleared& to = sm.cleared[(segs - 1) & 7];
#pragma unroll 1
                for (int r = half * 8; r < half * 8 + 8; ++r) {
                    const int tok = tl.t0 + r * 8;
                    // (a region that was not copied, on a bad page, has what lay there before)
                    if ((tl.ok >> r & 1u) && tok >= tl.all_lo && tok + 7 <= tl.all_hi) continue;
                    uint4* v = reinterpret_cast<uint4*>(vs + st * kTileBytes + r * kRegionBytes);
                    uint4 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = v[i * 32 + lane];
                    uint32_t any = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) any |= all_ones(x[i].x) | all_ones(x[i].y) | all_ones(x[i].z) | all_ones(x[i].w);
                    if (__builtin_expect(__any_sync(0xffffffffu, any != 0), 0)) {
                        // the region's tokens that some row sees (the segment's rows outlive its tiles), and those found
                        uint32_t seen = 0, found = 0;
                        for (int j = lane; j < NB && (tl.ok >> r & 1u); j += 32)
                            if (tl.rows >> j & 1u) {
                                const int pos = sm.rows[(segs - 1) & (kRowSegs - 1)][j];
                                const int a = p.window > 0 ? min(max(max(0, pos - p.window + 1) - tok, 0), 8) : 0, z = min(max(pos - tok + 1, 0), 8);
                                if (z > a) seen |= (1u << z) - (1u << a);
                            }
#pragma unroll 1
                        for (int i = 0; i < 16; ++i) {
                            uint32_t* at = reinterpret_cast<uint32_t*>(v + (i >> 2) * 32 + lane) + (i & 3);
                            const uint32_t bad = all_ones(*at);
                            if (bad == 0) continue;
                            *at &= ~((bad >> 15) * 0xffffu);
                            found |= 1u << (((i >> 2 & 1) * 32 + lane) >> 3);
                        }
                        found = __reduce_or_sync(0xffffffffu, found) & __reduce_or_sync(0xffffffffu, seen);
                        if (found && lane == 0) {
                            atomicMin(&to.lo, tok + __ffs(found) - 1);
                            atomicMax(&to.hi, tok + 31 - __clz(found));
                            atomicOr(&to.runs, 1ull << (tok >> 7 & 63));
                        }
                    }
                }
            }
            fence_proxy_async();
            if (t + 1 < run && failed(wait(&sm.kfull[(t + 1) % kStagesK], (uint32_t)(((t + 1) / kStagesK) & 1)))) break;
            __syncwarp();
            if (lane == 0) arrive(&sm.go[st]);
        }
    } else {
        // ---------------- softmax: 64 keys of a head row to a thread
        const int w = (warp - kSoftWarp) >> 3, half = warp >> 2 & 1 ^ 1;  // row tile, half of its keys (and of O's dims)
        const int r = tid & 127, hr = w * 128 + r, j = w * RB + r / HQ;  // head row in the row tile, in the block; row of the block
        const int pair = 1 + w * 4 + (warp & 3);                      // barrier of this warp and that of the other half
        const uint32_t lanes = tc::taddr(tmem, (warp & 3) * 32, 0);
        const uint32_t s_at = lanes + 128u * w + 64u * half, p_at = lanes + 128u * w + 32u * half, o_at = lanes + 256u + 128u * w + 64u * half;
        float neg_m = INFINITY, l = 0.0f;  // (l: of this thread's keys)
        int pos = -1, lo = 0;              // the row's first and last token; pos < 0: none, -1: padding, -2: out of range
        bool begun = false;                // the row tile has had a tile of the segment
        uint32_t e_note = 0;               // of the segment
        int e_g = 0, e_n0 = 0, e_last = 0;

        // x of the row's two threads through op, in both.
        auto joined = [&](float x, auto op) {
            if (half == 1) sm.part[hr] = x;
            group_or(pair, 64, false);
            if (half == 0) sm.part[hr] = x = op(x, sm.part[hr]);
            group_or(pair, 64, false);
            return half == 0 ? x : sm.part[hr];
        };
        // A wait that gave up must end the pair's two warps together: they tell each other at their barrier.
        auto waited = [&](uint64_t* bar, uint32_t parity) {
            if (__all_sync(0xffffffffu, wait(bar, parity) && *reinterpret_cast<volatile int*>(&sm.fail) == 0)) return true;
            if (lane == 0) give_up();
            return false;
        };

        // The output, or partial state, of segment number i.
        auto epilogue = [&](int i) {
            if (group_or(pair, 64, !waited(&sm.obar[w], (uint32_t)(i & 1)))) return false;
            tc::fence_after_sync();
            const bool whole = (e_note & kWhole) != 0, begins = (e_note & kBegins) != 0;
            const Cleared& cl = sm.cleared[i & 7];
            const int first = max(cl.lo, lo), last = min(cl.hi, pos);
            l = joined(l, [](float a, float b) { return a + b; });
            float f = l == 0.0f ? 0.0f : 1.0f / l;
            const int64_t at = (int64_t)(e_n0 + j) * p.Hq + (int64_t)e_g * HQ + r % HQ;
            float* st = p.states + ((int64_t)2 * blockIdx.x + (begins ? 1 : 0)) * kStateFloats;
            if (!whole && half == 0) *reinterpret_cast<float2*>(st + 2 * hr) = make_float2(-neg_m, l);
            if (whole && p.gate != nullptr && pos >= 0) f *= 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[at])));
#pragma unroll 1
            for (int c = 64 * half; c < 64 * half + 64; c += 32) {
                float o[32];
                __syncwarp();
                tc::ld32(lanes + 256u + 128u * w + c, o);
#pragma unroll
                for (int d = 0; d < 32; ++d) o[d] = l == 0.0f ? 0.0f : o[d] * f;
                if (whole && pos != -1) {
#pragma unroll
                    for (int d = 0; d < 32; d += 16) {
                        uint32_t u[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) u[x] = pack_bf16x2(o[d + 2 * x], o[d + 2 * x + 1]);
                        store32(p.out + at * 128 + c + d, u);
                    }
                } else if (!whole) {  // CTAs share the item; each leaves its state, which the join kernel reads
#pragma unroll
                    for (int d = 0; d < 32; d += 8) {
                        uint32_t u[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) u[x] = __float_as_uint(o[d + x]);
                        store32(st + 512 + ((c + d) >> 3) * 2048 + hr * 8, u);
                    }
                }
            }
            const bool adds = first <= last && l != 0.0f;
            if (__builtin_expect(__any_sync(0xffffffffu, adds), 0))
                add_not_finite(p, cl, adds ? p.row_seq[e_n0 + j] : -1, e_g, 64 * half, first, last, p.out + at * 128 + 64 * half,
                               whole ? nullptr : st + 512 + 8 * half * 2048 + hr * 8);
            if (!whole && begins && hr == 0 && half == 0) p.shared_items[blockIdx.x] = make_int4(e_n0, e_g, (int)blockIdx.x, e_last);
            return true;
        };

        for (int t = 0, segs = 0; t < run; ++t) {
            const bool bad = !waited(&sm.sbar[w], (uint32_t)(t & 1));
            tc::fence_after_sync();
            const Tile& tl = sm.ring[t & (kRing - 1)];
            const uint32_t note = tl.note;
            const bool idle = (note & kIdle << w) != 0;
            uint32_t x[2][32];  // the half row of S
            tc::get32(s_at, x[0]);
            tc::get32(s_at + 32, x[1]);
            if (note & kFirst) {
                e_note = note, e_g = tl.g, e_n0 = tl.n0, e_last = tl.last;
                pos = sm.rows[segs & (kRowSegs - 1)][j];
                lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
                if (pos == -2) raise_status(p.status, kDevRange);
                neg_m = INFINITY, l = 0.0f, begun = false;
            }
            tc::got32(x[0]);
            tc::got32(x[1]);
            if (idle) {
                if (group_or(pair, 64, bad)) break;
            } else {
                if (!(note & kAll)) {  // the columns that the row sees: from .. to - 1, of readable regions
                    int from = 0, to = 0;
                    if (pos >= 0 && (tl.rows >> j & 1u)) {
                        from = min(max(lo - tl.t0 - 64 * half, 0), 64);
                        to = min(max(pos - tl.t0 + 1 - 64 * half, 0), 64);
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t okr = tl.ok >> (8 * half + 4 * c) & 15u;
                        const uint32_t below = to - 32 * c >= 32 ? ~0u : (1u << max(to - 32 * c, 0)) - 1u;
                        const uint32_t under = from - 32 * c >= 32 ? ~0u : (1u << max(from - 32 * c, 0)) - 1u;
                        const uint32_t mask = below & ~under & ((okr * 0x00204081u & 0x01010101u) * 0xffu);
                        if (__any_sync(0xffffffffu, mask != ~0u))
#pragma unroll
                            for (int d = 0; d < 32; ++d) x[c][d] = mask >> d & 1u ? x[c][d] : 0xff800000u;
                    }
                }
                // the largest logit of the thread's keys (in log2 units); the running maximum follows the row's when it is
                // passed by more than the slack, which rescales l and O
                float m2[2] = {__uint_as_float(x[0][0]), __uint_as_float(x[0][1])};
#pragma unroll
                for (int d = 2; d < 62; d += 4) {
                    m2[0] = max3(m2[0], __uint_as_float(x[d / 32][d % 32]), __uint_as_float(x[(d + 1) / 32][(d + 1) % 32]));
                    m2[1] = max3(m2[1], __uint_as_float(x[(d + 2) / 32][(d + 2) % 32]), __uint_as_float(x[(d + 3) / 32][(d + 3) % 32]));
                }
                float mx = max3(m2[0], m2[1], fmaxf(__uint_as_float(x[1][30]), __uint_as_float(x[1][31]))) * p.scale_log2;
                auto passed = [&](float m) { return m > kSlack - neg_m || (neg_m == INFINITY && m > -INFINITY); };
                // (the pair's barrier also stands between the reads of S and P, which takes its place)
                tc::fence_before_sync();
                if (__builtin_expect(group_or(pair, 64, passed(mx) || bad), 0)) {
                    if (group_or(pair, 64, bad)) break;
                    mx = joined(mx, [](float a, float b) { return fmaxf(a, b); });
                    float f = 1.0f;
                    if (passed(mx)) {
                        f = ex2(-neg_m - mx);
                        l *= f;
                        neg_m = -mx;
                    }
                    if (begun) {
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            float o[16];
                            tc::ld16(o_at + c, o);
#pragma unroll
                            for (int d = 0; d < 16; ++d) o[d] *= f;
                            tc::st16(o_at + c, o);
                        }
                    }
                }
                tc::fence_after_sync();
                // weights, 8 bits each in bf16 as V is
                const float2 scale = both(p.scale_log2), nm = both(neg_m == INFINITY ? 0.0f : neg_m);
                float2 sum[2] = {both(0.0f), both(0.0f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int d = 0; d < 32; d += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(x[c][d]), __uint_as_float(x[c][d + 1])), scale, nm);
                        const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
                        sum[d / 2 & 1] = add2(sum[d / 2 & 1], e2);
                        pk[d / 2] = pack_bf16x2(e2.x, e2.y);
                    }
                    tc::st16u(p_at + 16 * c, pk);
                }
                begun = true;
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive(&sm.pbar[w]);
            if ((note & kLast) && !epilogue(segs++)) break;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::dealloc(tmem, kCols);
}

template <int HQ>
cudaError_t launch_heads(const PagedAttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         int num_sms, cudaStream_t stream, bool pdl) {
    using S = Shape<HQ>;
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        static_assert(kSmem<S> <= 227 * 1024, "shared memory");
        return cudaFuncSetAttribute(paged_chunk_bf16_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem<S>);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms < kChunkMaxCtas ? num_sms : kChunkMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem<S>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, paged_chunk_bf16_kernel<S>, qmap, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_join<S>(p, num_sms, cfg);
}

}  // namespace

cudaError_t launch_paged_chunk_bf16(const PagedAttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap,
                                    const CUtensorMap& vmap, int num_sms, cudaStream_t stream, bool pdl) {
    switch (p.Hq / p.G) {
        case 4: return launch_heads<4>(p, qmap, kmap, vmap, num_sms, stream, pdl);
        case 8: return launch_heads<8>(p, qmap, kmap, vmap, num_sms, stream, pdl);
        case 16: return launch_heads<16>(p, qmap, kmap, vmap, num_sms, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace step5
