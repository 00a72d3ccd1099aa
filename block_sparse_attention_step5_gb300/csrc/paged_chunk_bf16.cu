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
// A softmax thread owns a head row: it takes the row of S into registers whole, so that its maximum and its weights
// need neither another thread nor a second look at S.  The row tiles take turns: while one's softmax runs,
// the tensor core has the other's two products (1,024 cycles for 128 rows against 128 keys).
//
// Unseen values.  A weight of zero must meet a finite value, but a page may hold anything where a row does not look.
// Where some row of the block does not see some key of the tile (its edges), two warps look the tile of V over, clear what
// is not finite, and note the tokens it was found at; the rows that see one of those tokens take it up again at
// their end, from the page itself.
//
// Work.  As over the e4m3 pages: the tiles of all (block of rows, group) items are laid end to end, each CTA takes an equal
// run, and a second kernel joins the items that CTAs share.
#include <type_traits>

#include "paged_blocks.cuh"

namespace step5 {

namespace {

constexpr int kMmaWarp = 8, kLoadWarp = 9, kCheckWarp = 10;  // (two of the last)
constexpr int kThreads = 12 * 32;
constexpr int kRing = 8;
constexpr int kStagesK = 3, kStagesV = 2;
constexpr uint32_t kRegionBytes = 2048, kTileBytes = kTile * kRegionBytes, kQBytes = 128 * 256;
constexpr uint32_t kSmem = 1024 + 2 * kQBytes + (kStagesK + kStagesV) * kTileBytes;
constexpr uint32_t kCols = 512;                 // S of both row tiles (P in the first half of each), O of both
constexpr uint32_t kIdescQk = tc::instr_desc(tc::kFmtBF16, false, false, 128, 128);
constexpr uint32_t kIdescPv = tc::instr_desc(tc::kFmtBF16, false, true, 128, 128);
constexpr float kSlack = 8.0f;                  // log2 units a weight may lie above the running maximum

// A tile as the copying warp leaves it for the others.
struct Tile {
    uint64_t rows;       // the block's rows that the tile's sequence is of
    uint32_t ok;         // regions that can be read and hold keys
    int t0;              // first token
    uint32_t note;       // 1: the segment's first tile, 2: its last, 4: every row of the block but padding sees every key
    int b, g, n0;        // sequence, group, first row of the block
};

// Tokens of a segment whose values are not finite and were cleared, the first and the last (none: hi < lo).
struct Cleared {
    int lo, hi;
};

// What dims c .. c + 31 hold among tokens lo .. hi of sequence b: masks of infinities of either sign (a NaN is both).
__device__ __noinline__ uint2 not_finite(const PagedAttnParams& p, int b, int g, int c, int lo, int hi) {
    uint32_t pos = 0, neg = 0;
    for (int t = lo; t <= hi; ++t) {
        const int64_t row = page_row(p.pages, p.G, b, g, t);
        if (row < 0) continue;
        const uint4* v = reinterpret_cast<const uint4*>(p.v_pages + row * 256 + c * 2);
        for (int i = 0; i < 4; ++i) {
            const uint4 x = v[i];
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
            for (int y = 0; y < 8; ++y) {
                const uint32_t u = xs[y >> 1] >> (16 * (y & 1)) & 0xffffu;
                if ((u & 0x7f80u) != 0x7f80u) continue;
                if ((u & 0x7fu) || !(u & 0x8000u)) pos |= 1u << (8 * i + y);
                if ((u & 0x7fu) || (u & 0x8000u)) neg |= 1u << (8 * i + y);
            }
        }
    }
    return make_uint2(pos, neg);
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_bf16_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, PagedAttnParams p) {
    constexpr int HQ = S::HQ, RB = S::RB, NB = S::NB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw, 1024);
    uint8_t* qs = smem;                               // [row tile][half of the dims][128 head rows][128 B], 128-byte swizzle
    uint8_t* ks = qs + 2 * kQBytes;                   // [stage][16 regions][half][8 tokens][128 B], swizzled
    uint8_t* vs = ks + kStagesK * kTileBytes;
    __shared__ __align__(8) uint64_t kfull[kStagesK], kempty[kStagesK], vfull[kStagesV], vempty[kStagesV], vok[kStagesV], sbar[2],
        pbar[2], obar[2], qbar, fbar;
    __shared__ __align__(16) Tile ring[kRing];
    __shared__ Cleared s_cleared[8];                  // of segment i % 8
    __shared__ BlockRunSmem<kThreads> rs;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int blocks = (p.N + NB - 1) / NB;

    if (tid == 0) {
        prefetch_tmap(&qmap);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        for (int i = 0; i < kStagesK; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < kStagesV; ++i) {
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 1);
            mbar_init(&vok[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sbar[i], 2);
            mbar_init(&pbar[i], 4);
            mbar_init(&obar[i], 2);
        }
        mbar_init(&qbar, 1);
        mbar_init(&fbar, 1);
        fence_mbar_init();
        s_fail = 0;
    }
    if (tid < 8) s_cleared[tid] = Cleared{INT32_MAX, -1};
    if (warp == kMmaWarp) tc::alloc(&s_tmem, kCols);
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) p.shared_items[blockIdx.x].w = -1;
    const BlockRun of = take_run<S, kThreads>(p, rs, reinterpret_cast<int*>(smem));  // (nothing is copied yet)
    const int64_t of_group = of.of_group, total = of.total, per = of.per, start = of.start;
    fence_proxy_async();  // (the copies write where the tiles' numbers were)
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    const int run = (int)(start < total ? min(per, total - start) : 0);
    const int blk0 = rs.blk, off0 = rs.off, g0 = run ? (int)(start / of_group) : 0;

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
        // ---------------- copies: K_0, q, K_1, V_0, K_2, V_1, ..., q of a new block behind the last product of the one before;
        // lane l looks up region l % 16 of tile l / 16 of two
        const int k = p.box_regions, q = lane & 15;
        Walk<S> w{};
        Segment s{g0, blk0, off0, 0, 0};
        int left = run, seg_left = 0, issued_k = 0, issued_v = 0, segs = 0;
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
                if (t >= kStagesK && !wait(&kempty[t % kStagesK], (uint32_t)((t / kStagesK - 1) & 1))) ok = false;
                if (failed(ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int t0 = (w.r0 + w.at * kTile) * 8;
                    const bool all = oks == 0xffffu && w.rows == w.valid && w.bad == 0 && t0 >= w.max_lo && t0 + 127 <= w.min_hi;
                    Tile& tl = ring[t & (kRing - 1)];
                    tl.rows = w.rows;
                    tl.ok = oks;
                    tl.t0 = t0;
                    tl.note = (first ? 1u : 0u) | (seg_left == 0 ? 2u : 0u) | (all ? 4u : 0u);
                    tl.b = w.b;
                    tl.g = s.g;
                    tl.n0 = s.blk * NB;
                }
                const int n0 = s.blk * NB, g = s.g;
                if (seg_left == 0) {  // on to the next item
                    s.off = 0;
                    ++s.blk;
                }
                if (!(lane < 16 && (q & (k - 1)) == 0)) nrow = -1;
                const uint32_t have = __ballot_sync(0xffffffffu, nrow >= 0);
                __syncwarp();
                const int st = t % kStagesK;
                if (lane == 0) mbar_arrive_expect_tx(&kfull[st], (uint32_t)__popc(have) * kRegionBytes * k);
                __syncwarp();
                if (nrow >= 0) tma_load_4d(ks + st * kTileBytes + q * kRegionBytes, &kmap, &kfull[st], 0, 0, 0, nrow >> 3);
                issued_k = t + 1;
                if (first && t == 0 && lane == 0) {
                    mbar_arrive_expect_tx(&qbar, 2 * kQBytes);
                    tma_load_4d(qs, &qmap, &qbar, 0, g * HQ, n0, 0);
                    tma_load_4d(qs + kQBytes, &qmap, &qbar, 0, g * HQ, n0 + RB, 0);
                }
                if (first) ++segs;
                __syncwarp();
            }
            if (t > 0) {
                const int v = t - 1, st = v % kStagesV;
                if (v >= kStagesV && !wait(&vempty[st], (uint32_t)((v / kStagesV - 1) & 1))) ok = false;
                if (failed(ok)) {
                    ok = false;
                    break;
                }
                const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
                if (lane == 0) mbar_arrive_expect_tx(&vfull[st], (uint32_t)__popc(have) * kRegionBytes * k);
                __syncwarp();
                if (row >= 0) tma_load_4d(vs + st * kTileBytes + q * kRegionBytes, &vmap, &vfull[st], 0, 0, 0, row >> 3);
                issued_v = t;
                if (t < run && first) {  // the products of the block before have read its q
                    if (!wait(&kempty[v % kStagesK], (uint32_t)((v / kStagesK) & 1))) ok = false;
                    if (failed(ok)) {
                        ok = false;
                        break;
                    }
                    const Tile& tl = ring[t & (kRing - 1)];
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&qbar, 2 * kQBytes);
                        tma_load_4d(qs, &qmap, &qbar, 0, tl.g * HQ, tl.n0, 0);
                        tma_load_4d(qs + kQBytes, &qmap, &qbar, 0, tl.g * HQ, tl.n0 + RB, 0);
                    }
                    __syncwarp();
                }
            }
            row = nrow;
        }
        if (!ok && lane == 0) {  // let the copies issued land (bounded) before the shared memory goes away
            give_up();
            for (int i = max(0, issued_k - kStagesK); i < issued_k; ++i) wait(&kfull[i % kStagesK], (uint32_t)((i / kStagesK) & 1));
            for (int i = max(0, issued_v - kStagesV); i < issued_v; ++i) wait(&vfull[i % kStagesV], (uint32_t)((i / kStagesV) & 1));
            if (segs > 0) wait(&qbar, (uint32_t)((segs - 1) & 1));
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------- products, of the row tiles in turn: P V of a tile, then Q K of the next, whose S takes P's
        // place (products of one thread run in order).  Behind a segment's last tile q changes: both
        // P V go first.
        const uint32_t k_addr = smem_u32(ks), v_addr = smem_u32(vs), q_addr = smem_u32(qs);
        bool ok = true;
        int segs = 0;
        auto check = [&](bool waited) {
            ok = __all_sync(0xffffffffu, waited) && ok;
            if (!ok && lane == 0) give_up();
            return ok;
        };
        uint32_t note = 0;  // of the tile whose Q K was issued last
        auto qk = [&](int w, int t) {
            const int st = t % kStagesK;
            if (w == 0) {
                if (!check(wait(&kfull[st], (uint32_t)((t / kStagesK) & 1)))) return;
                note = __shfl_sync(0xffffffffu, ring[t & (kRing - 1)].note, 0);
                if ((note & 1u) && !check(wait(&qbar, (uint32_t)(segs++ & 1)))) return;
            }
            tc::fence_after_sync();
            const uint64_t db = tc::smem_desc(k_addr + (uint32_t)st * kTileBytes, 16, kRegionBytes, tc::kSwizzle128);
            const uint64_t da = tc::smem_desc(q_addr + (uint32_t)w * kQBytes, 16, 1024, tc::kSwizzle128);
            if (elect()) {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 16 dims each
                    tc::mma_f16(tmem + 128u * w, da + (i < 4 ? 2 * i : (kQBytes >> 5) + 2 * (i - 4)), db + (i < 4 ? 2 * i : 64 + 2 * (i - 4)),
                                kIdescQk, i > 0);
                arrive(&sbar[w]);  // (hands the tile's ring entry on, which came with its K)
                tc::commit(&sbar[w]);
                if (w == 1) tc::commit(&kempty[st]);
            }
            __syncwarp();
        };
        auto pv = [&](int w, int t, uint32_t of) {
            const int st = t % kStagesV;
            if (w == 0 && !check(wait(&vfull[st], (uint32_t)((t / kStagesV) & 1)) && wait(&vok[st], (uint32_t)((t / kStagesV) & 1)))) return;
            if (!check(wait(&pbar[w], (uint32_t)(t & 1)))) return;
            tc::fence_after_sync();
            const uint64_t db = tc::smem_desc(v_addr + (uint32_t)st * kTileBytes, 1024, kRegionBytes, tc::kSwizzle128);
            if (elect()) {
#pragma unroll
                for (int i = 0; i < 8; ++i)  // 16 keys each
                    tc::mma_f16_ts(tmem + 256u + 128u * w, tmem + 128u * w + 8u * i, db + (2 * kRegionBytes >> 4) * i, kIdescPv, !(of & 1u) || i > 0);
                if (of & 2u) {
                    arrive(&obar[w]);  // (hands the checking warps' notes on)
                    tc::commit(&obar[w]);
                }
                if (w == 1) tc::commit(&vempty[st]);
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
    } else if (warp >= kCheckWarp) {
        // ---------------- V of the tiles that not every row sees whole: what is not finite becomes zero, and is noted
        const int half = warp - kCheckWarp;  // regions 8 half .. 8 half + 7
        int segs = 0;
        for (int t = 0; t < run; ++t) {
            const int st = t % kStagesV;
            if (failed(wait(&vfull[st], (uint32_t)((t / kStagesV) & 1)))) break;
            const Tile& tl = ring[t & (kRing - 1)];
            const uint32_t note = tl.note;
            if (note & 1u) {
                // (segment i - 5's notes have been read: its successors' tiles have been worked on)
                if (half == 0 && lane == 0) s_cleared[(segs + 3) & 7] = Cleared{INT32_MAX, -1};
                ++segs;
            }
            if (!(note & 4u)) {
                Cleared& to = s_cleared[(segs - 1) & 7];
                uint4* v = reinterpret_cast<uint4*>(vs + st * kTileBytes + half * 8 * kRegionBytes);
#pragma unroll 4
                for (int i = 0; i < 32; ++i) {  // a quarter of a region each
                    const uint4 x = v[i * 32 + lane];
                    uint32_t xs[4] = {x.x, x.y, x.z, x.w}, bad[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) bad[y] = ((xs[y] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // an exponent of all ones
                    if (__builtin_expect((bad[0] | bad[1] | bad[2] | bad[3]) != 0, 0)) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) xs[y] &= ~((bad[y] >> 15) * 0xffffu);
                        v[i * 32 + lane] = make_uint4(xs[0], xs[1], xs[2], xs[3]);
                        const int r = half * 8 + (i >> 2), tok = tl.t0 + r * 8 + (((i & 1) * 32 + lane) >> 3);
                        if (tl.ok >> r & 1u) {
                            atomicMin(&to.lo, tok);
                            atomicMax(&to.hi, tok);
                        }
                    }
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(&vok[st]);
        }
    } else {
        // ---------------- softmax: a head row to a thread
        const int w = warp >> 2, r = tid & 127, j = w * RB + r / HQ;  // row tile, head row in it, row of the block
        const uint32_t lanes = tc::taddr(tmem, (warp & 3) * 32, 0);
        const uint32_t s_at = lanes + 128u * w, o_at = lanes + 256u + 128u * w;
        float neg_m = INFINITY, l = 0.0f;
        Row row{-1, -1, 0};
        Segment s{g0, blk0, off0, 0, 0}, e = s;  // e: the segment that the epilogue is of
        int64_t e_begin = 0;                     // its item's first tile, among all
        Row e_row = row;
        int t = 0, segs = 0;
        bool ok = true;

        // The output, or partial state, of segment number i, e.
        auto epilogue = [&](int i) {
            if (failed(wait(&obar[w], (uint32_t)(i & 1)))) {
                ok = false;
                return;
            }
            tc::fence_after_sync();
            const bool whole = e.n == e.nt;
            const Cleared cl = s_cleared[i & 7];
            const int lo = max(cl.lo, e_row.lo), hi = e_row.b >= 0 ? min(cl.hi, e_row.pos) : -1;
            float f = l == 0.0f ? 0.0f : 1.0f / l;
            const int hr = w * 128 + r;
            const int64_t at = (int64_t)(e.blk * NB + j) * p.Hq + (int64_t)e.g * HQ + r % HQ;
            float* st = p.states + ((int64_t)2 * blockIdx.x + (e_begin >= start ? 1 : 0)) * kStateFloats;
            if (!whole) *reinterpret_cast<float2*>(st + 2 * hr) = make_float2(-neg_m, l);
            if (whole && p.gate != nullptr && e_row.b >= 0) f *= 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[at])));
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                __syncwarp();
                tc::ld32(o_at + c, o);
#pragma unroll
                for (int d = 0; d < 32; ++d) o[d] = l == 0.0f ? 0.0f : o[d] * f;
                if (__builtin_expect(lo <= hi && l != 0.0f, 0)) {
                    const uint2 m = not_finite(p, e_row.b, e.g, c, lo, hi);
#pragma unroll
                    for (int d = 0; d < 32; ++d) {
                        if (m.x >> d & 1u) o[d] += INFINITY;
                        if (m.y >> d & 1u) o[d] -= INFINITY;
                    }
                }
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
            if (!whole && e_begin >= start && tid == 0)
                p.shared_items[blockIdx.x] = make_int4(e.blk * NB, e.g, (int)blockIdx.x, (int)((e_begin + e.nt - 1) / per));
        };

        for (int left = run; left > 0 && ok;) {
            {
                Walk<S> walk;
                if (!next(s, walk, left)) {
                    if (lane == 0) give_up();
                    ok = false;
                    break;
                }
            }
            row = row_at(p, s.blk * NB + j);
            if (row.b == -2) raise_status(p.status, kDevRange);
            if (segs > 0) epilogue(segs - 1);
            if (!ok) break;
            e = s;
            e_row = row;
            e_begin = start + (run - left) - s.off;
            ++segs;
            left -= s.n;
            s.off = 0;
            ++s.blk;
            neg_m = INFINITY, l = 0.0f;
            for (int i = 0; i < e.n; ++i, ++t) {
                if (failed(wait(&sbar[w], (uint32_t)(t & 1)))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                uint32_t x[4][32];  // the row of S
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::get32(s_at + 32 * c, x[c]);
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::got32(x[c]);
                const Tile& tl = ring[t & (kRing - 1)];
                if (!(tl.note & 4u)) {  // the columns that the row sees: from .. to - 1, of readable regions
                    int from = 0, to = 0;
                    if (row.b >= 0 && (tl.rows >> j & 1u)) {
                        from = min(max(row.lo - tl.t0, 0), 128);
                        to = min(max(row.pos - tl.t0 + 1, 0), 128);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t okr = tl.ok >> (4 * c) & 15u;
                        const uint32_t below = to - 32 * c >= 32 ? ~0u : (1u << max(to - 32 * c, 0)) - 1u;
                        const uint32_t under = from - 32 * c >= 32 ? ~0u : (1u << max(from - 32 * c, 0)) - 1u;
                        const uint32_t mask = below & ~under & ((okr * 0x00204081u & 0x01010101u) * 0xffu);
#pragma unroll
                        for (int d = 0; d < 32; ++d) x[c][d] = mask >> d & 1u ? x[c][d] : 0xff800000u;
                    }
                }
                // the row's largest logit in the tile (in log2 units); the running maximum follows it when it is
                // passed by more than the slack, which rescales l and O
                float m4[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    m4[c] = __uint_as_float(x[c][0]);
#pragma unroll
                    for (int d = 1; d < 31; d += 2) m4[c] = max3(m4[c], __uint_as_float(x[c][d]), __uint_as_float(x[c][d + 1]));
                    m4[c] = fmaxf(m4[c], __uint_as_float(x[c][31]));
                }
                const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * p.scale_log2;
                const bool up = mx > kSlack - neg_m || (neg_m == INFINITY && mx > -INFINITY);
                if (__builtin_expect(__any_sync(0xffffffffu, up), 0)) {
                    float f = 1.0f;
                    if (up) {
                        f = ex2(-neg_m - mx);
                        l *= f;
                        neg_m = -mx;
                    }
                    if (i > 0) {
#pragma unroll 1
                        for (int c = 0; c < 128; c += 16) {
                            float o[16];
                            tc::ld16(o_at + c, o);
#pragma unroll
                            for (int d = 0; d < 16; ++d) o[d] *= f;
                            tc::st16(o_at + c, o);
                        }
                    }
                }
                // weights, 8 bits each in bf16 as V is: P takes the first half of S's place
                const float2 scale = both(p.scale_log2), nm = both(neg_m == INFINITY ? 0.0f : neg_m);
                float2 sum[2] = {both(0.0f), both(0.0f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int d = 0; d < 32; d += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(x[c][d]), __uint_as_float(x[c][d + 1])), scale, nm);
                        const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
                        sum[d / 2 & 1] = add2(sum[d / 2 & 1], e2);
                        pk[d / 2] = pack_bf16x2(e2.x, e2.y);
                    }
                    tc::st16u(s_at + 16 * c, pk);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
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
cudaError_t launch_heads(const PagedAttnParams& p, const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                         int num_sms, cudaStream_t stream, bool pdl) {
    using S = Shape<HQ>;
    static std::atomic<uint64_t> attr_set{0};
    cudaError_t e = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(paged_chunk_bf16_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
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
