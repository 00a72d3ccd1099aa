// paged_chunk.cu -- attention over the e4m3 paged cache for launches whose sequences have several
// rows (prompt chunks, drafts): the rows of a sequence share its keys.
//
//   s_t = softmax_scale (q . kcode_t) kscale(region of t),  p = softmax(s),  out = sum_t p_t vscale vcode_t
//
// A CTA takes two tiles of 128 head rows (128 / HQ consecutive rows of the call, HQ query heads each)
// against 128 keys at a time:
//
//   S [128 head rows x 128 keys]  = q_hi . K^T + q_lo . K^T   (kind::f8f6f4, K's codes as they lie in the cache)
//   O [128 head rows x 128 dims] += P . V                     (kind::f16, P from tensor memory)
//
// With head rows on the M side a softmax thread owns a row: its maximum, sum and rescaling need no
// other thread.  q is two e4m3 numbers, hi + lo (lo the rounding of what hi leaves: exact for values
// above 2^-9 of the head's largest, off by at most 2^-17 of that below), which share an accumulator.
// V's codes are turned into f16 (exact) by four warps, once for both row tiles, and P is f16 (11
// bits), so that weights keep 2^-11 and a range of 2^-33: e4m3 parts of P would cost more here, where
// P is as large as S.  One tile of rows and keys is 512 cycles of tensor core in either product (an
// e4m3 product runs twice as fast as f16 and is done twice), which would bound the kernel with the
// softmax of one row tile under the products of the other.
//
// Scales.  kscale goes into the factor of the exponent, eight keys at a time; vscale joins the
// weight, relative to a power of two (vref) not below any vscale that the row has seen; the row sum
// takes the weight without it.
//
// Work.  As in the kernel for single rows, the tiles of all (block of rows, group) items are laid end
// to end and each CTA takes an equal run; a second kernel joins the items that CTAs share.  A block's
// rows may belong to several sequences: its tiles are those of each sequence in turn, with the other
// rows masked.
//
// What it takes, with 4 KV groups of 8 heads and pages of 64 tokens, join included:
//   2,048 rows behind 2,048 tokens    138 us  1.03e11 flop (at 1,899 TFLOP/s: 54 us)
//   2,048 rows, window of 512 tokens   61 us  1.7e10 flop (9 us)
// A tile of keys takes its two row tiles 2.5 us: maximum 1,050, weights 1,400, the products and the
// waits around them 2,200 cycles (1,024 of tensor core; the first product alone reads shared memory
// at its full rate, which the copies and V's conversion share).  Around the tiles: start 4 us, q 3 us
// and epilogue 2 us for each part of an item, join 3 us.
#include <type_traits>

#include "paged_blocks.cuh"

namespace step5 {

namespace {

constexpr int kConvWarp = 8, kMmaWarp = 12, kLoadWarp = 13;
constexpr int kThreads = 14 * 32;
constexpr int kRing = 8;
constexpr uint32_t kKv8Bytes = 128 * 128, kV16Bytes = 2 * kKv8Bytes, kQPartBytes = 128 * 128;
// q: two row tiles x two parts; two tiles of K, of V as it lies in the cache, and of V in f16
constexpr uint32_t kSmem = 1024 + 4 * kQPartBytes + 2 * kKv8Bytes + 2 * kKv8Bytes + 2 * kV16Bytes;
constexpr uint32_t kCols = 512;                 // S of both row tiles (P in the first half of each), O of both
constexpr uint32_t kIdescQk = tc::instr_desc(tc::kFmtE4M3, false, false, 128, 128);
constexpr uint32_t kIdescPv = tc::instr_desc(tc::kFmtF16, false, true, 128, 128);
constexpr float kSlack = 6.0f;                  // log2 units a weight may lie above the running maximum
constexpr float kPTop = 256.0f;                 // P = p 2^8 vscale / vref <= 2^14
// vref is at least this, so that kPTop / vref is finite: a weight times the smallest vscale, 2^-126, is then P itself, whose finest
// step is 2^-24
constexpr float kVrefMin = 0x1p-118f;

// A tile as the copying warp leaves it for the others.
struct Tile {
    float ks[kTile], vs[kTile];
    uint64_t rows;       // the block's rows that the tile's sequence is of
    uint32_t ok;         // regions that can be read and hold keys
    int t0;              // first token
    int lo, hi;          // the pass's first and last token
    uint32_t note;       // 1: the segment's first tile, 2: its last, 4: every row of the block but padding sees every key
    float vmax;          // largest vscale of the ok regions
    int n0;              // first row of the block
};

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       PagedAttnParams p) {
    constexpr int HQ = S::HQ, RB = S::RB, NB = S::NB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw, 1024);
    uint8_t* qs = smem;                               // [row tile][part][128 rows][128 B], 128-byte swizzle
    uint8_t* k8 = qs + 4 * kQPartBytes;               // [2][128 keys][128 B], swizzled by the copy
    uint8_t* v8 = k8 + 2 * kKv8Bytes;
    uint8_t* v16 = v8 + 2 * kKv8Bytes;                // [2][half of the dims][128 keys][64 dims], swizzled
    __shared__ __align__(8) uint64_t kfull[2], kempty[2], vfull[2], vempty[2], cfull[2], cempty[2], sbar[2], pbar[2], obar[2], qbar[2],
        fbar;
    __shared__ __align__(16) Tile ring[kRing];
    __shared__ unsigned long long s_nan[8][128];      // of segment i % 8: the rows that see a NaN in this dim
    __shared__ uint32_t s_any_nan[8];
    __shared__ int2 s_seen[4][NB];                    // by converting warp: the rows' first and last token
    __shared__ BlockRunSmem<kThreads> rs;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int blocks = (p.N + NB - 1) / NB;

    if (tid == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kempty[i], 1);
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 4);
            mbar_init(&cfull[i], 4);
            mbar_init(&cempty[i], 1);
            mbar_init(&sbar[i], 2);
            mbar_init(&pbar[i], 4);
            mbar_init(&obar[i], 2);
            mbar_init(&qbar[i], 4);
        }
        mbar_init(&fbar, 1);
        fence_mbar_init();
        s_fail = 0;
    }
    for (int i = tid; i < 8 * 128; i += kThreads) s_nan[i >> 7][i & 127] = 0;
    if (tid < 8) s_any_nan[tid] = 0;
    if (warp == kMmaWarp) tc::alloc(&s_tmem, kCols);
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) p.shared_items[blockIdx.x].w = -1;

    const BlockRun of = take_run<S, kThreads>(p, rs, reinterpret_cast<int*>(smem));  // (nothing is copied yet)
    const int64_t per = of.per, start = of.start;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const int run = of.run, blk0 = rs.blk, off0 = rs.off, g0 = of.g0;

    // Every role walks the run's segments alike: item (group, block), tiles off .. off + n - 1 of it.
    // next() returns false when there is none (the rows have changed under the kernel).
    struct Segment {
        int g, blk, off, n, nt;
    };
    auto next = [&](Segment& s, Walk<S>& w, int left) -> bool {
        for (;;) {
            if (s.blk >= blocks) {
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
        atomicExch(&s_fail, 1);
    };
    auto failed = [&](bool ok) {  // for a whole warp
        if (!__all_sync(0xffffffffu, ok && *reinterpret_cast<volatile int*>(&s_fail) == 0)) {
            if (lane == 0) give_up();
            return true;
        }
        return false;
    };

    if (run == 0) {
        // nothing to do
    } else if (warp == kLoadWarp) {
        // ---------------- copies: K_0, K_1, V_0, K_2, V_1, ...; lane l looks up region l % 16 of tile l / 16 of two
        const int k = p.box_regions, q = lane & 15;
        Walk<S> w{};
        Segment s{g0, blk0, off0, 0, 0};
        int left = run, seg_left = 0, issued_k = 0, issued_v = 0;
        int b_row = -1, n_row = -1, batch = -1, done = 0;
        uint32_t b_seen = 0, n_seen = 0;  // lanes whose region some row sees
        float b_ks = 0.0f, b_vs = 0.0f, n_ks = 0.0f, n_vs = 0.0f;
        bool ok = true;
        auto look = [&](int of, int steps) {
            const int r = w.r0 + (of * 2 + (lane >> 4)) * kTile + q;
            if (steps & 1) {
                n_row = -1;
                n_seen = __ballot_sync(0xffffffffu, w.sees(r));
                if (n_seen >> (lane & ~(k - 1)) & ((1u << k) - 1u)) {  // (some region of its box)
                    n_row = (int)page_row(p.pages, p.G, w.b, s.g, r * 8);
                    if (n_row < 0) raise_status(p.status, kDevRange);
                }
            }
            if (steps & 2) {
                n_ks = n_vs = 0.0f;
                if (n_row >= 0) {
                    n_ks = p.k_scales[n_row >> 3];
                    n_vs = p.v_scales[n_row >> 3];
                }
            }
        };
        int row = -1;  // of the tile whose V is next
        for (int t = 0; t <= run; ++t) {
            int nrow = -1;
            if (t < run) {
                const bool first = seg_left == 0;
                if (first) {
                    if (!next(s, w, left)) {
                        ok = false;
                        break;
                    }
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
                    if (done != 3) look(w.at >> 1, 3 & ~done);
                    batch = w.at >> 1;
                    b_row = n_row, b_seen = n_seen, b_ks = n_ks, b_vs = n_vs, done = 0;
                    if ((batch + 1) * 2 < w.tiles && (w.at & 1) == 0) {
                        look(batch + 1, 1);
                        done = 1;
                    }
                } else if ((batch + 1) * 2 < w.tiles) {
                    look(batch + 1, 3 & ~done);
                    done = 3;
                }
                const int from = (w.at & 1) * 16 + q;
                nrow = __shfl_sync(0xffffffffu, b_row, from);
                const float ks = __shfl_sync(0xffffffffu, b_ks, from), vs = __shfl_sync(0xffffffffu, b_vs, from);
                bool good = nrow >= 0 && (b_seen >> from & 1u);
                if (good && !(scale_ok(ks) && scale_ok(vs))) {
                    raise_status(p.status, kDevRange);
                    good = false;
                }
                const uint32_t oks = __ballot_sync(0xffffffffu, good) & 0xffffu;
                const uint32_t vmax = __reduce_max_sync(0xffffffffu, good ? __float_as_uint(vs) : 0u);
                if (t >= 2 && !wait(&kempty[t & 1], (uint32_t)(((t - 2) >> 1) & 1))) ok = false;
                if (failed(ok)) {
                    ok = false;
                    break;
                }
                Tile& tl = ring[t & (kRing - 1)];
                if (lane < 16) {
                    tl.ks[q] = good ? ks : 0.0f;
                    tl.vs[q] = good ? vs : 0.0f;
                }
                if (lane == 0) {
                    const int t0 = (w.r0 + w.at * kTile) * 8;
                    const bool all = oks == 0xffffu && w.rows == w.valid && w.bad == 0 && t0 >= w.max_lo && t0 + 127 <= w.min_hi;
                    tl.rows = w.rows;
                    tl.ok = oks;
                    tl.t0 = t0;
                    tl.lo = w.lo;
                    tl.hi = w.hi;
                    tl.note = (first ? 1u : 0u) | (seg_left == 0 ? 2u : 0u) | (all ? 4u : 0u);
                    tl.vmax = __uint_as_float(vmax);
                    tl.n0 = s.blk * NB;
                }
                if (seg_left == 0) {  // on to the next item
                    s.off = 0;
                    ++s.blk;
                }
                if (!(lane < 16 && (q & (k - 1)) == 0)) nrow = -1;
                const uint32_t have = __ballot_sync(0xffffffffu, nrow >= 0);
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&kfull[t & 1], (uint32_t)__popc(have) * 1024u * k);
                __syncwarp();
                if (nrow >= 0) tma_load_2d(k8 + (t & 1) * kKv8Bytes + q * 1024, &kmap, &kfull[t & 1], 0, nrow);
                issued_k = t + 1;
            }
            if (t > 0) {
                const int v = t - 1;
                if (v >= 2 && !wait(&vempty[v & 1], (uint32_t)(((v - 2) >> 1) & 1))) ok = false;
                if (failed(ok)) {
                    ok = false;
                    break;
                }
                const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
                if (lane == 0) mbar_arrive_expect_tx(&vfull[v & 1], (uint32_t)__popc(have) * 1024u * k);
                __syncwarp();
                if (row >= 0) tma_load_2d(v8 + (v & 1) * kKv8Bytes + q * 1024, &vmap, &vfull[v & 1], 0, row);
                issued_v = t;
            }
            row = nrow;
        }
        if (!ok && lane == 0) {  // let the copies issued land (bounded) before the shared memory goes away
            give_up();
            for (int i = max(0, issued_k - 2); i < issued_k; ++i) wait(&kfull[i & 1], (uint32_t)((i >> 1) & 1));
            for (int i = max(0, issued_v - 2); i < issued_v; ++i) wait(&vfull[i & 1], (uint32_t)((i >> 1) & 1));
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------- products, of the row tiles in turn: P V of a tile, then Q K of the next, whose S takes P's
        // place (products of one thread run in order).  Behind a segment's last tile q changes: both
        // P V go first.
        const uint32_t k_addr = smem_u32(k8), v_addr = smem_u32(v16), q_addr = smem_u32(qs);
        bool ok = true;
        int segs = 0;
        auto check = [&](bool waited) {
            ok = __all_sync(0xffffffffu, waited) && ok;
            if (!ok && lane == 0) give_up();
            return ok;
        };
        uint32_t note = 0;  // of the tile whose Q K was issued last
        auto qk = [&](int w, int t) {
            if (w == 0) {
                if (!check(wait(&kfull[t & 1], (uint32_t)((t >> 1) & 1)))) return;
                note = __shfl_sync(0xffffffffu, ring[t & (kRing - 1)].note, 0);
                if (note & 1u) ++segs;
            }
            if ((note & 1u) && !check(wait(&qbar[w], (uint32_t)((segs - 1) & 1)))) return;
            tc::fence_after_sync();
            const uint64_t db = tc::smem_desc(k_addr + (uint32_t)(t & 1) * kKv8Bytes, 16, 1024, tc::kSwizzle128);
            const uint64_t da = tc::smem_desc(q_addr + 2u * w * kQPartBytes, 16, 1024, tc::kSwizzle128);
            if (elect()) {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 32 dims of q_hi, then of q_lo
                    tc::mma_f8(tmem + 128u * w, da + (i < 4 ? 0u : kQPartBytes >> 4) + 2u * (i & 3), db + 2u * (i & 3), kIdescQk, i > 0);
                arrive(&sbar[w]);  // (hands the tile's ring entry on, which came with its K)
                tc::commit(&sbar[w]);
                if (w == 1) tc::commit(&kempty[t & 1]);
            }
            __syncwarp();
        };
        auto pv = [&](int w, int t, uint32_t of) {
            if (w == 0 && !check(wait(&cfull[t & 1], (uint32_t)((t >> 1) & 1)))) return;
            if (!check(wait(&pbar[w], (uint32_t)(t & 1)))) return;
            tc::fence_after_sync();
            const uint64_t db = tc::smem_desc(v_addr + (uint32_t)(t & 1) * kV16Bytes, kKv8Bytes, 1024, tc::kSwizzle128);
            if (elect()) {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 16 keys each
                    tc::mma_f16_ts(tmem + 256u + 128u * w, tmem + 128u * w + 8u * i, db + 128u * i, kIdescPv, !(of & 1u) || i > 0);
                if (of & 2u) {
                    arrive(&obar[w]);  // (hands the converting warps' notes on)
                    tc::commit(&obar[w]);
                }
                if (w == 1) tc::commit(&cempty[t & 1]);
            }
            __syncwarp();
        };
        qk(0, 0);
        if (ok) qk(1, 0);
        for (int t = 0; t < run && ok; ++t) {
            const uint32_t of = note;
            const bool more = t + 1 < run, turn = (of & 2u) != 0;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (ok) pv(w, t, of);
                if (ok && more && !turn) qk(w, t + 1);
            }
            if (ok && more && turn) {
                qk(0, t + 1);
                if (ok) qk(1, t + 1);
            }
        }
        if (!ok) {  // the products issued end before their memory goes away
            if (elect()) tc::commit(&fbar);
            __syncwarp();
            wait(&fbar, 0);
        }
        __syncwarp();
    } else if (warp >= kConvWarp) {
        // ---------------- V's codes to f16: a key to a thread.  In a tile of which some row does not see some key, NaN codes
        // become zero (the cache may hold anything there, and a zero weight must meet a finite
        // value), noted for the rows that see them.
        const int cw = warp - kConvWarp, key = cw * 32 + lane;
        int segs = 0;
        for (int t = 0; t < run; ++t) {
            bool ok = wait(&vfull[t & 1], (uint32_t)((t >> 1) & 1));
            if (t >= 2) ok = ok && wait(&cempty[t & 1], (uint32_t)(((t - 2) >> 1) & 1));
            if (failed(ok)) break;
            const Tile& tl = ring[t & (kRing - 1)];
            const uint32_t note = tl.note;
            if (note & 1u) {  // the segment's rows
                // (segment i - 5's notes have been read: its successors' tiles have been worked on)
                if (cw == 0) {
                    for (int i = lane; i < 128; i += 32) s_nan[(segs + 3) & 7][i] = 0;
                    if (lane == 0) s_any_nan[(segs + 3) & 7] = 0;
                }
                ++segs;
                __syncwarp();
                for (int i = lane; i < NB; i += 32) {
                    const Row r = row_at(p, tl.n0 + i);
                    s_seen[cw][i] = make_int2(r.lo, r.pos);
                }
                __syncwarp();
            }
            const uint4* src = reinterpret_cast<const uint4*>(v8 + (t & 1) * kKv8Bytes + key * 128);
            uint8_t* dst = v16 + (t & 1) * kV16Bytes + key * 128;
            const int sw = key & 7;
            auto widen = [&](int c, const uint4& x) {  // dims 16 c .. 16 c + 15: chunks 2 (c % 4) and the next of half c / 4
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(xs[i] & 0xffffu), __NV_E4M3);
                    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(xs[i] >> 16), __NV_E4M3);
                    const __half2 a2(a), b2(b);
                    h[2 * i] = *reinterpret_cast<const uint32_t*>(&a2);
                    h[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                uint8_t* to = dst + (c >> 2) * kKv8Bytes;
                *reinterpret_cast<uint4*>(to + (((2 * (c & 3)) ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(to + (((2 * (c & 3) + 1) ^ sw) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            };
            if (note & 4u) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) widen(c, src[c ^ sw]);
            } else {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    const uint4 x = src[c ^ sw];
                    uint32_t xs[4] = {x.x, x.y, x.z, x.w}, bad[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) bad[i] = ((xs[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // 0x7f, 0xff
                    if (__builtin_expect((bad[0] | bad[1] | bad[2] | bad[3]) != 0, 0)) {
                        const int tok = tl.t0 + key;
                        unsigned long long seen = 0;
                        if (tl.ok >> (key >> 3) & 1u)
                            for (uint64_t m = tl.rows; m; m &= m - 1) {
                                const int2 s = s_seen[cw][__ffsll((long long)m) - 1];
                                if (tok >= s.x && tok <= s.y) seen |= m & (0 - m);
                            }
                        if (seen) s_any_nan[(segs - 1) & 7] = 1;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            xs[i] &= ~((bad[i] >> 7) * 0xffu);
                            for (uint32_t m = seen ? bad[i] : 0u; m; m &= m - 1)
                                atomicOr(&s_nan[(segs - 1) & 7][c * 16 + i * 4 + ((__ffs(m) - 1) >> 3)], seen);
                        }
                    }
                    widen(c, make_uint4(xs[0], xs[1], xs[2], xs[3]));
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                arrive(&vempty[t & 1]);
                arrive(&cfull[t & 1]);
            }
        }
    } else {
        // ---------------- softmax: a head row to a thread
        const int w = warp >> 2, r = tid & 127, j = w * RB + r / HQ;  // row tile, head row in it, row of the block
        const uint32_t lanes = tc::taddr(tmem, (warp & 3) * 32, 0);
        const uint32_t s_at = lanes + 128u * w, o_at = lanes + 256u + 128u * w;
        float neg_m = INFINITY, l = 0.0f, vref = 0.0f, vinv = 0.0f, cq = 0.0f;
        Row row{-1, -1, 0};
        Walk<S> walk{};
        Segment s{g0, blk0, off0, 0, 0}, e = s;  // e: the segment that the epilogue is of
        int64_t e_begin = 0;                     // its item's first tile, among all
        Row e_row = row;
        int t = 0, segs = 0;
        bool ok = true;

        // The warp's 32 head rows, eight lanes of 16 dims to each; the next eight rows are on their
        // way meanwhile.
        auto build_q = [&] {
            const int l8 = lane & 7, hr0 = (warp & 3) * 32 + (lane >> 3);
            const uint32_t rows_ok = __ballot_sync(0xffffffffu, row.b >= 0);
            const uint16_t* src = p.q + ((int64_t)(s.blk * NB + w * RB) * p.Hq + (int64_t)s.g * HQ) * 128 + l8 * 16;
            uint4 nx[2][2];
            auto ask = [&](int i0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int hr = hr0 + i0 + 4 * i;
                    nx[i][0] = nx[i][1] = make_uint4(0, 0, 0, 0);
                    if (rows_ok >> (i0 + 4 * i + (lane >> 3)) & 1u) {
                        const uint4* at = reinterpret_cast<const uint4*>(src + ((int64_t)(hr / HQ) * p.Hq + hr % HQ) * 128);
                        nx[i][0] = at[0];
                        nx[i][1] = at[1];
                    }
                }
            };
            ask(0);
#pragma unroll 1
            for (int i0 = 0; i0 < 32; i0 += 8) {
                const uint4 x[2][2] = {{nx[0][0], nx[0][1]}, {nx[1][0], nx[1][1]}};
                if (i0 < 24) ask(i0 + 8);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int hr = hr0 + i0 + 4 * i;
                    const uint32_t xs[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                    uint32_t a2 = 0;
#pragma unroll
                    for (int y = 0; y < 8; ++y) a2 = __vmaxu2(a2, xs[y] & 0x7fff7fffu);
#pragma unroll
                    for (int d = 4; d; d >>= 1) a2 = __vmaxu2(a2, __shfl_xor_sync(0xffffffffu, a2, d));
                    const uint32_t a = max(a2 & 0xffffu, a2 >> 16);
                    // q * 2^(7 - e) is below 2^8 for the largest |q|, whose exponent is e
                    const int ex = a == 0 ? 0 : max((int)(a >> 7) - 127, -100);
                    const float up = __uint_as_float((uint32_t)(min(7 - ex, 120) + 127) << 23);
                    const float c = a < 0x7f80u ? p.scale_log2 / up : __int_as_float(0x7fc00000);
                    const float mine = __shfl_sync(0xffffffffu, c, (lane & 3) * 8);
                    if (lane >> 2 == (i0 >> 2) + i) cq = mine;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float2 v2 = mul2(make_float2(bf16_lo(xs[y]), bf16_hi(xs[y])), both(up));
                        const __half2 v = __float22half2_rn(v2);
                        const uint32_t h = last_part(v);
                        const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
                        const uint32_t l = last_part(__hsub2(v, __half2(back)));
                        hi[y >> 1] = y & 1 ? __byte_perm(hi[y >> 1], h, 0x5410) : h;
                        lo[y >> 1] = y & 1 ? __byte_perm(lo[y >> 1], l, 0x5410) : l;
                    }
                    uint8_t* to = qs + 2 * w * kQPartBytes + hr * 128 + ((l8 ^ (hr & 7)) << 4);
                    *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(to + kQPartBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(&qbar[w]);
        };

        // Scales O by f, this thread's row's factor.
        auto rescale = [&](float f) {
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                uint32_t u[32];
                tc::ld32(o_at + c, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
                tc::st32(o_at + c, u);
            }
        };

        // The output, or partial state, of segment number i, e.
        auto epilogue = [&](int i) {
            if (failed(wait(&obar[w], (uint32_t)(i & 1)))) {
                ok = false;
                return;
            }
            tc::fence_after_sync();
            const bool any_nan = s_any_nan[i & 7] != 0, whole = e.n == e.nt;
            float f = l == 0.0f ? 0.0f : (1.0f / kPTop) / l;  // (times vref below: their product may underflow)
            const int hr = w * 128 + r;
            const int64_t at = (int64_t)(e.blk * NB + j) * p.Hq + (int64_t)e.g * HQ + r % HQ;
            float* st = p.states + ((int64_t)2 * blockIdx.x + (e_begin >= start ? 1 : 0)) * kStateFloats;
            if (!whole) *reinterpret_cast<float2*>(st + 2 * hr) = make_float2(-neg_m, l);
            if (whole && p.gate != nullptr && e_row.b != -1) f *= 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[at])));
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                __syncwarp();
                tc::ld32(o_at + c, o);
#pragma unroll
                for (int d = 0; d < 32; ++d) o[d] = l == 0.0f ? 0.0f : o[d] * f * vref;
                if (any_nan)
#pragma unroll
                    for (int d = 0; d < 32; ++d)
                        if (s_nan[i & 7][c + d] >> j & 1u) o[d] = __int_as_float(0x7fc00000);
                if (whole && e_row.b != -1) {
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
            if (e.n != e.nt && e_begin >= start && tid == 0)
                p.shared_items[blockIdx.x] = make_int4(e.blk * NB, e.g, (int)blockIdx.x, (int)((e_begin + e.nt - 1) / per));
        };

        for (int left = run; left > 0 && ok;) {
            if (!next(s, walk, left)) {
                if (lane == 0) give_up();
                ok = false;
                break;
            }
            row = row_at(p, s.blk * NB + j);
            if (row.b == -2) raise_status(p.status, kDevRange);
            build_q();
            if (segs > 0) epilogue(segs - 1);
            if (!ok) break;
            e = s;
            e_row = row;
            e_begin = start + (run - left) - s.off;
            ++segs;
            left -= s.n;
            s.off = 0;
            ++s.blk;
            neg_m = INFINITY, l = vref = vinv = 0.0f;
            for (int i = 0; i < e.n; ++i, ++t) {
                if (failed(wait(&sbar[w], (uint32_t)(t & 1)))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const Tile& tl = ring[t & (kRing - 1)];
                // the columns that the row sees, unless every row sees all: from .. to - 1, of
                // readable regions
                const bool all = (tl.note & 4u) != 0;
                int from = 0, to = 0;
                if (!all && row.b >= 0 && (tl.rows >> j & 1u)) {
                    from = min(max(row.lo - tl.t0, 0), 128);
                    to = min(max(row.pos - tl.t0 + 1, 0), 128);
                }
                // those of columns c .. c + 31 as a mask
                auto seen = [&](int c) {
                    const uint32_t okr = tl.ok >> (c >> 3) & 15u;
                    const uint32_t below = to - c >= 32 ? ~0u : (1u << max(to - c, 0)) - 1u;
                    const uint32_t under = from - c >= 32 ? ~0u : (1u << max(from - c, 0)) - 1u;
                    return below & ~under & ((okr * 0x00204081u & 0x01010101u) * 0xffu);
                };
                // the row's largest logit in the tile (in log2 units); the running maximum follows it
                // when it is passed by more than the slack, which rescales l and O
                float mx = -INFINITY;
                uint32_t x[32];  // columns of S
                auto largest = [&](int c, const uint32_t(&x)[32], auto edge) {
                    const uint32_t mask = decltype(edge)::value ? seen(c) : ~0u;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float v[8];
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            v[d] = __uint_as_float(x[8 * g + d]);
                            if constexpr (decltype(edge)::value) v[d] = mask >> (8 * g + d) & 1u ? v[d] : -INFINITY;
                        }
                        const float m8 = fmaxf(max3(max3(v[0], v[1], v[2]), v[3], v[4]), max3(v[5], v[6], v[7]));
                        mx = fmaxf(mx, m8 * tl.ks[c / 8 + g]);  // (ks > 0 where the region is readable; -inf * 0 is no maximum)
                    }
                };
                // (loops, not unrolled further: straight code for a whole tile ran 20 % slower, short
                // of instructions)
                auto all_largest = [&](auto edge) {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        tc::get32(s_at + c, x);
                        tc::got32(x);
                        largest(c, x, edge);
                    }
                };
                if (all)
                    all_largest(std::false_type{});
                else
                    all_largest(std::true_type{});
                mx *= cq;
                const bool up = mx > kSlack - neg_m || (neg_m == INFINITY && mx > -INFINITY), higher = tl.vmax > vref;
                if (__builtin_expect(__any_sync(0xffffffffu, up || higher), 0)) {
                    float f = 1.0f;
                    if (up) {
                        f = ex2(-neg_m - mx);
                        l *= f;
                        neg_m = -mx;
                    }
                    if (higher) {  // vref follows the largest vscale that the row itself sees
                        float v = tl.vmax;
                        if (!all) {
                            const uint32_t regs = from < to ? (2u << ((to - 1) >> 3)) - (1u << (from >> 3)) : 0u;
                            v = 0.0f;
#pragma unroll 1
                            for (uint32_t m = regs; m; m &= m - 1) v = fmaxf(v, tl.vs[__ffs(m) - 1]);  // (0 where it cannot be read)
                        }
                        if (v > vref) {
                            const uint32_t u = __float_as_uint(v);
                            const float p2 = fmaxf(__uint_as_float((u & 0x7f800000u) + ((u & 0x7fffffu) ? 0x800000u : 0u)), kVrefMin);
                            f *= vref / p2;
                            vref = p2;
                            vinv = 1.0f / p2;
                        }
                    }
                    if (i > 0 && __any_sync(0xffffffffu, f != 1.0f)) rescale(f);
                }
                // weights: P takes the first half of S's place, behind the columns already read
                const float vtop = vinv * kPTop;
                float2 sum = both(0.0f);
                auto weights = [&](int c, const uint32_t(&x)[32], auto edge) {
                    uint32_t pk[16];
                    const uint32_t mask = decltype(edge)::value ? seen(c) : ~0u;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int reg = c / 8 + g;
                        // (at most kPTop where the row sees the region; a weight of 0 must meet a finite factor)
                        float vr = tl.vs[reg] * vtop;
                        if constexpr (decltype(edge)::value) vr = fminf(vr, kPTop);
                        const float2 f = both(tl.ks[reg] * cq), vf = both(vr), nm = both(neg_m);
#pragma unroll
                        for (int d = 0; d < 8; d += 2) {
                            float2 y = fma2(make_float2(__uint_as_float(x[8 * g + d]), __uint_as_float(x[8 * g + d + 1])), f, nm);
                            if constexpr (decltype(edge)::value) {
                                y.x = mask >> (8 * g + d) & 1u ? y.x : -INFINITY;
                                y.y = mask >> (8 * g + d + 1) & 1u ? y.y : -INFINITY;
                            }
                            const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
                            sum = add2(sum, e2);
                            const __half2 h = __float22half2_rn(mul2(e2, vf));
                            pk[4 * g + d / 2] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
                    tc::st16u(s_at + c / 2, pk);
                };
                auto all_weights = [&](auto edge) {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        tc::get32(s_at + c, x);
                        tc::got32(x);
                        weights(c, x, edge);
                    }
                };
                if (all)
                    all_weights(std::false_type{});
                else
                    all_weights(std::true_type{});
                l += sum.x + sum.y;
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(&pbar[w]);
            }
        }
        if (ok) epilogue(segs - 1);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::dealloc(tmem, kCols);
}

template <int HQ>
cudaError_t launch_heads(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int num_sms,
                         cudaStream_t stream, bool pdl) {
    using S = Shape<HQ>;
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(paged_chunk_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms < kChunkMaxCtas ? num_sms : kChunkMaxCtas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, paged_chunk_kernel<S>, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_join<S>(p, num_sms, cfg);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int num_sms,
                               cudaStream_t stream, bool pdl) {
    static_assert((size_t)kChunkMaxCtas * 2 * kStateFloats <= kPagedStateFloats, "workspace");
    switch (p.Hq / p.G) {
        case 4: return launch_heads<4>(p, kmap, vmap, num_sms, stream, pdl);
        case 8: return launch_heads<8>(p, kmap, vmap, num_sms, stream, pdl);
        case 16: return launch_heads<16>(p, kmap, vmap, num_sms, stream, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace step5
