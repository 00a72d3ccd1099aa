// paged_attention_bf16.cu -- attention over the bf16 paged cache, rows on their own: every token of a causal window,
// or the picked regions plus the row's own.
//
//   s_t = softmax_scale (q . k_t),  p = softmax(s),  out = sum_t p_t v_t
//
// As over the e4m3 pages, 128 keys are the M side of both products and the H heads of a row the small one,
//
//   S^T [128 keys x H]    = K_tile [128 x 128 dims]        . q^T            (two TMEM buffers)
//   O^T [128 dims x 2 H] += V_tile^T [128 dims x 128 keys] . (p parts)^T
//
// with bf16 operands as the cache has them.  A weight has 8 bits in bf16; its rounding error goes along as a second part, more columns of
// the small side, which cost nothing, so 16 bits of each weight meet V.  A region (8 tokens x 256 B) lands as two swizzle atoms,
// [half of the dims][8 tokens][128 B], from one box of a 4-D view of the pool (64 dims x 8 tokens x 2 halves x regions): the K-major
// operand of the first product and the MN-major one of the second.
//
// The split of the work, the roles of the warps and the join are those of the kernel over the e4m3 pages.
#include "paged_items.cuh"

namespace step5 {

namespace {

constexpr int kSoft = 128;           // softmax threads
constexpr int kThreads = kSoft + 64 + 64;
constexpr int kQkWarp = 4, kLoadWarp = 6, kLoadWarps = 2;  // (the second product's warp is 5)
constexpr int kRing = 8;             // tiles whose masks are in shared memory
constexpr uint32_t kRegionBytes = 2048, kSlotBytes = kTile * kRegionBytes;
constexpr float kSlack = 8.0f;       // log2 units a tile's maximum may pass the running one by

template <int H_, bool PICKS_, int CTAS_>
struct Shape {
    static constexpr int H = H_;                       // query heads of a group
    static constexpr bool PICKS = PICKS_;
    static constexpr int kCtas = CTAS_;                // per SM
    static constexpr int kSlots = CTAS_ == 1 ? 6 : 3;
    static_assert(kSlots <= 6, "the barriers of copies and the ring are reused after 4 and 8 tiles");
    static constexpr int NS = 16;                      // columns of S: the heads
    static constexpr int NO = 2 * H < 16 ? 16 : 2 * H; // columns of O: the weights' two parts
    static constexpr uint32_t kCols = 64;
    static constexpr uint32_t kQBytes = NS * 256, kPBytes = 128 * NO * 2;
    static constexpr uint32_t kPGroup = 16 * NO;       // bytes of 8 keys of P
    static constexpr uint32_t kSmem = 1024 + kSlots * kSlotBytes + kQBytes + 2 * kPBytes;
    static constexpr uint32_t kIdesc1 = tc::instr_desc(tc::kFmtBF16, false, false, 128, NS);
    static constexpr uint32_t kIdesc2 = tc::instr_desc(tc::kFmtBF16, true, true, 128, NO);
    static constexpr int kState = H * 130;             // floats of a partial state: m[H], l[H], o[H][128]
    static_assert(2 * NS + NO <= (int)kCols, "tensor memory");
};

template <class S>
__global__ void __launch_bounds__(kThreads, S::kCtas)
    paged_attn_bf16_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      PagedAttnParams p) {
    constexpr int H = S::H;
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
    __shared__ int s_note[kRing];  // of a tile: MMA steps | first tile of a segment << 8
    __shared__ float red[3][4][H];
    __shared__ RunSmem<kThreads> rs;

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
    if (H < S::NS)  // q rows that no head fills (softmax threads, which fence them below)
        for (int i = tid; i < (S::NS - H) * 16; i += kSoft)
            if (tid < kSoft) {
                const int half = i / ((S::NS - H) * 8), r = i % ((S::NS - H) * 8);
                reinterpret_cast<uint4*>(qt + half * S::NS * 128 + H * 128)[r] = make_uint4(0, 0, 0, 0);
            }
    pdl_wait();
    pdl_launch_dependents();

    int64_t start, per;
    const bool few = take_run<PICKS, kThreads>(p, rs, start, per);
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
                    const int t0 = b_r * 8;
                    const int a = min(max(it.lo - t0, 0), 8), z = min(max(it.hi - t0 + 1, 0), 8);
                    const uint32_t mask = b_row >= 0 && z > a ? ((1u << z) - 1u) & ~((1u << a) - 1u) : 0u;
                    ring[t & (kRing - 1)][q] = mask | (b_row >= 0 ? 256u : 0u);
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
                    it = rs.it;
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
        Item it{}, done{};  // the segment's item; that of the segment before, for its epilogue
        int64_t done_begin = 0;
        bool whole = true, begins = true;  // it has the whole item, its first tile
        bool failed = false;
        int t = 0;  // tile of the run

        auto give_up = [&] {
            raise_status(p.status, kDevTimeout);
            atomicExch(&s_fail, 1);
        };

        // The item's heads, 16 lanes to each.
        auto build_q = [&] {
#pragma unroll
            for (int u0 = 0; u0 < H; u0 += 8) {
                const int u = u0 + (tid >> 4), d8 = tid & 15;
                if (H < 8 && u >= H) break;  // (whole warps)
                uint4 x = make_uint4(0, 0, 0, 0);
                if (it.b >= 0)
                    x = *reinterpret_cast<const uint4*>(p.q + (int64_t)it.n * p.q_stride + ((int64_t)it.g * H + u) * 128 + d8 * 8);
                *reinterpret_cast<uint4*>(qt + (d8 >> 3) * S::NS * 128 + u * 128 + (((d8 & 7) ^ (u & 7)) << 4)) = x;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive(&qbar);
        };

        // O of the segment that ended with tile t - 1, and its output or partial state.
        auto epilogue = [&] {
            const int tl = t - 1;
            float(&rd)[4][H] = red[2];
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
            float o[H], a[16];
            const uint32_t ob = lanes + 2 * S::NS;
            tc::ld16(ob, a);
            if constexpr (H == 16) {
                float b[16];
                tc::ld16(ob + 16, b);
#pragma unroll
                for (int h = 0; h < H; ++h) o[h] = a[h] + b[h];
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) o[h] = a[h] + a[H + h];
            }
            float L[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                L[h] = (rd[0][h] + rd[1][h]) + (rd[2][h] + rd[3][h]);
                o[h] = L[h] == 0.0f ? 0.0f : o[h] / L[h];
            }
            if (whole) {
                const int64_t at = (int64_t)done.n * p.Hq + (int64_t)done.g * H;
                if (p.gate != nullptr)
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        if (L[h] != 0.0f) o[h] = gated(p, at + h, o[h]);  // (zero stays zero)
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
                    p.shared_items[item0] = make_int4(done.n, done.g, rs.first, rs.last);
                else
                    p.shared_items[blockIdx.x] = make_int4(done.n, done.g, (int)blockIdx.x, (int)((done_begin + done.tiles - 1) / per));
            }
        };

        int nitem = item0, off = off0;
        for (int left = run; left > 0;) {
            it = rs.it;
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
            build_q();
            if (t > 0) epilogue();
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
#pragma unroll
            for (int h = 0; h < H / 2; ++h) {
                neg_m[h] = both(INFINITY);
                l_part[h] = both(0.0f);
            }
            for (int i = 0; i < seg; ++i, ++t) {
                // (tile t - 2's second product is done too: the first product of this one waited for it)
                bool w_ok = wait(&sbar[t & 1], (uint32_t)((t >> 1) & 1));
                tc::fence_after_sync();
                const uint32_t me = ring[t & (kRing - 1)][q];
                const bool sees = (me >> (key & 7) & 1u) != 0;
                // s[h] = q . k in log2 units, y[h] that less the running maximum
                float2 s[H / 2], y[H / 2];
                {
                    float x[16];
                    tc::ld16(lanes + (uint32_t)(S::NS * (t & 1)), x);
#pragma unroll
                    for (int h = 0; h < H; h += 2) s[h / 2] = mul2(make_float2(x[h], x[h + 1]), both(p.scale_log2));
                }
                float top = -INFINITY;
#pragma unroll
                for (int h = 0; h < H; h += 2) {
                    y[h / 2] = add2(s[h / 2], neg_m[h / 2]);
                    top = fmaxf(top, fmaxf(y[h / 2].x, y[h / 2].y));
                }
                // The running maxima move when a key passes one by more than the slack; l and O are rescaled
                // then.  Every softmax thread takes the same steps.
                if (!w_ok) give_up();
                if (__builtin_expect(group_or(1, kSoft, (sees && top > kSlack) || !w_ok), 0)) {
                    if (*reinterpret_cast<volatile int*>(&s_fail) != 0) failed = true;
                    float alpha[H];
                    int hidx = 0;
#pragma unroll
                    for (int h = 0; h < H; ++h) alpha[h] = sees ? (h & 1 ? s[h / 2].y : s[h / 2].x) : -INFINITY;
                    const float wmax = fold<H, 16>(alpha, lane, &hidx, Max{});
                    float(&rd)[4][H] = red[t & 1];
                    if ((lane & (32 / H - 1)) == 0) rd[warp][hidx] = wmax;
                    if (group_or(1, kSoft, failed)) {
                        failed = true;
                        break;
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
                    for (int h = 0; h < H; h += 2) y[h / 2] = add2(s[h / 2], neg_m[h / 2]);
                    if (i > 0) {
                        w_ok = wait(&obar[(t - 1) & 1], (uint32_t)(((t - 1) >> 1) & 1));
                        tc::fence_after_sync();
#pragma unroll
                        for (int c = 0; c < S::NO; c += 16) {
                            float o[16];
                            tc::ld16(lanes + 2 * S::NS + c, o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] *= alpha[(c + x) % H];
                            tc::st16(lanes + 2 * S::NS + c, o);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, !sees)) {  // (a key that is not seen may have anything for a score)
#pragma unroll
                    for (int h = 0; h < H / 2; ++h) y[h] = sees ? y[h] : both(-INFINITY);
                }
                // A weight in two bf16 parts: its first 8 bits, and the next 8.  The second is above zero where the weight
                // is (its last bit is set), so that an infinite value meets two positive numbers.
                uint32_t hi[H / 2], lo[H / 2];
#pragma unroll
                for (int h = 0; h < H; h += 2) {
                    const float2 w = make_float2(ex2(y[h / 2].x), ex2(y[h / 2].y));
                    l_part[h / 2] = add2(l_part[h / 2], w);
                    const uint32_t a = __float_as_uint(w.x), b = __float_as_uint(w.y);
                    hi[h / 2] = __byte_perm(a, b, 0x7632);
                    lo[h / 2] = pack_bf16x2(__uint_as_float(a | 1u) - __uint_as_float(a & 0xffff0000u),
                                            __uint_as_float(b | 1u) - __uint_as_float(b & 0xffff0000u));
                }
                uint8_t* pb = pt + (t & 1) * S::kPBytes + q * S::kPGroup + (key & 7) * 16;
                if constexpr (H == 4) {
                    *reinterpret_cast<uint4*>(pb) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                } else {
#pragma unroll
                    for (int x = 0; x < H / 8; ++x) {
                        *reinterpret_cast<uint4*>(pb + x * 128) = make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
                        *reinterpret_cast<uint4*>(pb + (H / 8 + x) * 128) =
                            make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
                    }
                }
                // a copied V row that the row does not see is zeroed: the cache may hold anything
                // there, and a zero weight must meet a finite value
                if (__builtin_expect((me & 256u) && !sees, 0)) {
                    const int slot = (t + 1 < run ? 2 * t + 2 : 2 * t + 1) % S::kSlots;
                    w_ok &= wait(&vfull[t & 3], (uint32_t)((t >> 2) & 1));
                    uint4* vr = reinterpret_cast<uint4*>(slots + slot * kSlotBytes + q * kRegionBytes + (key & 7) * 128);
#pragma unroll
                    for (int x = 0; x < 8; ++x) vr[x] = vr[64 + x] = make_uint4(0, 0, 0, 0);
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
    if (p.sel_ids == nullptr) return launch_shape<Shape<H, false, 1>>(p, kmap, vmap, num_sms, stream, pdl);
    // (16 heads' weights leave room for one CTA an SM)
    return launch_shape<Shape<H, true, H == 16 ? 1 : 2>>(p, kmap, vmap, num_sms, stream, pdl);
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
