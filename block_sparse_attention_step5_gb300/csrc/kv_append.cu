// kv_append.cu -- the rows' keys and values into the paged cache (bf16, or e4m3 with a scale for each
// region and KV group), with NEOX rotation of k (and of q) on the way.
//
// Rotation is the indexer's (x1 c - x2 s, x2 c + x1 s over pairs (i, i + rot / 2) from bf16 cos/sin,
// the exact sum rounded once to bf16).  A head vector is sixteen 16-byte chunks and eight lanes:
// since rot / 2 is a multiple of 8, a lane takes both chunks of its eight pairs (or two that are only
// copied), so nothing is exchanged between lanes and every access is 16 bytes.  The kernel moves
// bytes: bound by HBM for chunks (2,048 rows of 40 heads in bf16, 42 MB), by the latency of its three
// dependent loads for a decode row.
//
// In e4m3 a region's eight tokens share a scale, so one warp (four tokens of eight lanes, twice)
// takes all of the call's tokens of a region for one (group, k or v), from the first of them on (the
// leader: a row on a region's first token, or one that does not continue the row before):
//   s = max(the scale held, if the region holds earlier tokens; the smallest power of two
//           >= max |x| / 448; 2^-126),      code = e4m3(x / s).
// A power of two divides exactly, costs an e4m3 value no precision (it has an exponent of its own),
// and makes the rescaling of tokens already held exact unless they leave the normal range. Those are
// requantised only when a new token raises the scale.
//
// With 4 KV groups, 32 query heads and pages of 64 tokens: one bf16 row 2.1 us; 2,048 rows in bf16
// 10.7 us (42 MB, 4.0 TB/s; 6.2 us at the copy bandwidth; 8,192 warps, 1.7 of the GPU's fill); 16 e4m3
// rows 3.0 us; 4 x 1,021 rows in e4m3 16.5 us (80 MB, 4.9 TB/s; 11.8 us), the exact rotation keeping the
// issue slots 60 % busy.
#include "paged.cuh"

namespace step5 {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kSeenWords = 1024;  // of a bit for each sequence

// Two chunks (8 bf16 each) of a head vector.
struct Chunks {
    uint4 a, b;
};

// First chunk of lane l8 of a vector whose first 2 * half8 chunks are rotated, and the distance to
// its second.
__device__ __forceinline__ int first_chunk(int l8, int half8) { return l8 < half8 ? l8 : 2 * l8; }
__device__ __forceinline__ int second_chunk(int l8, int half8) { return l8 < half8 ? l8 + half8 : 2 * l8 + 1; }

// x c + y s, products exact in fp32, rounded to odd: of the two fp32 numbers around the exact sum the
// one with an odd last bit.  Its rounding to bf16 (16 bits shorter) is the exact sum's.
__device__ __forceinline__ float odd_sum(float x, float c, float y, float s) {
    const float xc = __fmul_rn(x, c), down = __fmaf_rd(y, s, xc), up = __fmaf_ru(y, s, xc);
    return (__float_as_uint(down) & 1u) ? down : up;
}

__device__ __forceinline__ uint32_t rotate2(uint32_t x, uint32_t y, uint32_t c, uint32_t s, bool first) {
    const float n = first ? -1.0f : 1.0f;
    return pack_bf16x2(odd_sum(bf16_lo(x), bf16_lo(c), bf16_lo(y), n * bf16_lo(s)),
                       odd_sum(bf16_hi(x), bf16_hi(c), bf16_hi(y), n * bf16_hi(s)));
}

__device__ __forceinline__ void rotate(Chunks& x, const uint4& c, const uint4& s) {
    const Chunks o = x;
    x.a = make_uint4(rotate2(o.a.x, o.b.x, c.x, s.x, true), rotate2(o.a.y, o.b.y, c.y, s.y, true),
                     rotate2(o.a.z, o.b.z, c.z, s.z, true), rotate2(o.a.w, o.b.w, c.w, s.w, true));
    x.b = make_uint4(rotate2(o.b.x, o.a.x, c.x, s.x, false), rotate2(o.b.y, o.a.y, c.y, s.y, false),
                     rotate2(o.b.z, o.a.z, c.z, s.z, false), rotate2(o.b.w, o.a.w, c.w, s.w, false));
}

// The largest finite |bf16| of two packed ones, as bits (NaN left out, infinity taken as the largest
// finite value).
__device__ __forceinline__ uint32_t amax2(uint32_t w) {
    const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
    return min(max(a <= 0x7f80u ? a : 0u, b <= 0x7f80u ? b : 0u), 0x7f7fu);
}
__device__ __forceinline__ uint32_t amax8(const uint4& x) {
    return max(max(amax2(x.x), amax2(x.y)), max(amax2(x.z), amax2(x.w)));
}

// The smallest power of two s >= 2^-126 with |x| <= 448 s = 1.75 * 2^8 s, x given as bf16 bits.
__device__ __forceinline__ float scale_for(uint32_t amax) {
    const int e = (int)(amax >> 7) - 8 + ((amax & 127u) > 96u ? 1 : 0);  // biased exponent of s
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
    auto two = [&](uint32_t w) {
        return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(w) * inv, bf16_hi(w) * inv), __NV_SATFINITE,
                                                  __NV_E4M3);
    };
    return make_uint2(two(x.x) | (two(x.y) << 16), two(x.z) | (two(x.w) << 16));
}

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float f) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 v = e4m3x2_to_f32x2((uint16_t)(codes >> (16 * i)));
        v.x *= f;
        v.y *= f;
        r |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (16 * i);
    }
    return r;
}

__device__ __forceinline__ bool two_power(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// Scales that this file writes are powers of two, by which everything above is exact but for the
// rounding to e4m3. A scale held may be another's: then quotients and products are rounded
// towards zero and made odd where that left something, and their rounding to e4m3 is the exact value's.
// (Calls, and loops that are not unrolled: inlined, this cost every append 0.4 us.)
__device__ __forceinline__ float odd_rest(float v, float rest) {
    return rest != 0.0f && fabsf(v) < 1024.0f ? __uint_as_float(__float_as_uint(v) | 1u) : v;
}
__device__ __noinline__ uint32_t encode2_by(uint32_t x, float s) {
    const float up = s < 1.0f ? 0x1p64f : 1.0f;  // (what a division leaves must not underflow)
    float q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = (i ? bf16_hi(x) : bf16_lo(x)) * up;
        q[i] = __fdiv_rz(a, s * up);
        q[i] = odd_rest(q[i], __fmaf_rn(-q[i], s * up, a));
    }
    return __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
}
__device__ __noinline__ uint32_t rescale4_by(uint32_t codes, float f) {
    uint32_t r = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const float2 v = e4m3x2_to_f32x2((uint16_t)(codes >> (16 * i)));
        const float x = __fmul_rz(v.x, f), y = __fmul_rz(v.y, f);
        r |= (uint32_t)__nv_cvt_float2_to_fp8x2(
                 make_float2(odd_rest(x, __fmaf_rn(v.x, f, -x)), odd_rest(y, __fmaf_rn(v.y, f, -y))), __NV_SATFINITE, __NV_E4M3)
             << (16 * i);
    }
    return r;
}

// Row vectors: q's heads, and in bf16 k's and v's too.  Four vectors of the row to a warp at a time,
// two times in flight: q, k and v are asked for before the row's position is known.
template <bool E4M3>
__device__ __forceinline__ void append_row(const AppendParams& p, uint32_t id, int lane) {
    const int n = (int)(id >> p.row_shift), part = (int)(id & ((1u << p.row_shift) - 1)), l8 = lane & 7;
    if (n >= p.N) return;
    const int half8 = p.rot >> 4, c0 = first_chunk(l8, half8) * 8, c1 = second_chunk(l8, half8) * 8;
    const bool turns = l8 < half8;
    const int nq = p.q ? p.Hq : 0, vectors = nq + (E4M3 ? 0 : 2 * p.G), step = 4 << p.row_shift;
    const int b = p.row_seq[n], pos = p.row_pos[n];
    const bool ok = b >= 0 && b < p.B && pos >= 0 && pos < p.pos_cap;
    if (!ok && b != -1 && part == 0 && lane == 0) raise_status(p.status, kDevRange);
    uint4 cs = make_uint4(0, 0, 0, 0), sn = cs;
    for (int v0 = part * 4 + (lane >> 3); v0 < vectors; v0 += 2 * step) {
        Chunks x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = v0 + i * step, j = v - nq;
            if (v >= vectors) continue;
            const uint16_t* src = v < nq ? p.q + n * p.q_stride + (int64_t)v * 128
                                         : (j < p.G ? p.k + n * p.k_stride + (int64_t)j * 128
                                                    : p.v + n * p.v_stride + (int64_t)(j - p.G) * 128);
            x[i].a = *reinterpret_cast<const uint4*>(src + c0);
            x[i].b = *reinterpret_cast<const uint4*>(src + c1);
        }
        if (!ok) return;
        if (turns) {
            cs = *reinterpret_cast<const uint4*>(p.cos + (int64_t)pos * (p.rot >> 1) + 8 * l8);
            sn = *reinterpret_cast<const uint4*>(p.sin + (int64_t)pos * (p.rot >> 1) + 8 * l8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = v0 + i * step, j = v - nq;
            if (v >= vectors) continue;
            uint16_t* dst = p.q_out + ((int64_t)n * p.Hq + v) * 128;
            if (!E4M3 && v >= nq) {
                const int64_t row = page_row(p.pages, p.G, b, j < p.G ? j : j - p.G, pos);
                if (row < 0) {
                    if (l8 == 0) raise_status(p.status, kDevRange);
                    continue;
                }
                dst = static_cast<uint16_t*>(j < p.G ? p.k_pages : p.v_pages) + row * 128;
            }
            if (turns && (v < nq || j < p.G)) rotate(x[i], cs, sn);
            *reinterpret_cast<uint4*>(dst + c0) = x[i].a;
            *reinterpret_cast<uint4*>(dst + c1) = x[i].b;
        }
    }
}

// The m tokens of the call from row n on (position pos of sequence b) that lie in one region, for one
// (group, k or v).
__device__ __forceinline__ void append_region(const AppendParams& p, int n, int m, int b, int pos, int g, bool is_v,
                                              int lane) {
    const int l8 = lane & 7, tok = lane >> 3, t0 = pos & 7;
    const int64_t row = page_row(p.pages, p.G, b, g, pos);
    if (row < 0) {
        if (lane == 0) raise_status(p.status, kDevRange);
        return;
    }
    float* scale_at = (is_v ? p.v_scales : p.k_scales) + (row >> 3);
    uint8_t* codes = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + (row - t0) * 128;
    float held = 0.0f;  // read and written by the first lane alone
    if (t0 > 0 && lane == 0) held = *scale_at;
    const int half8 = p.rot >> 4, c0 = first_chunk(l8, half8) * 8, c1 = second_chunk(l8, half8) * 8;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const uint16_t* src = (is_v ? p.v : p.k) + n * stride + (int64_t)g * 128;
    Chunks x[2];
    uint4 cs[2], sn[2];
    const bool turns = !is_v && l8 < half8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = tok + 4 * i;
        x[i].a = x[i].b = cs[i] = sn[i] = make_uint4(0, 0, 0, 0);
        if (t < m) {
            x[i].a = *reinterpret_cast<const uint4*>(src + t * stride + c0);
            x[i].b = *reinterpret_cast<const uint4*>(src + t * stride + c1);
            if (turns) {
                const int64_t at = (int64_t)(pos + t) * (p.rot >> 1) + 8 * l8;
                cs[i] = *reinterpret_cast<const uint4*>(p.cos + at);
                sn[i] = *reinterpret_cast<const uint4*>(p.sin + at);
            }
        }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (turns) rotate(x[i], cs[i], sn[i]);
        amax = max(amax, max(amax8(x[i].a), amax8(x[i].b)));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    held = __shfl_sync(0xffffffffu, held, 0);
    float s = scale_for(amax);
    if (t0 > 0) {
        if (!scale_ok(held)) {
            if (lane == 0) raise_status(p.status, kDevRange);
        } else if (held >= s) {
            s = held;
        } else {
            const float f = held / s;  // (exact: s is a power of two)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (tok + 4 * i >= t0) continue;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint2* at = reinterpret_cast<uint2*>(codes + (tok + 4 * i) * 128 + (c ? c1 : c0));
                    const uint2 w = *at;
                    *at = two_power(f) ? make_uint2(rescale4(w.x, f), rescale4(w.y, f))
                                       : make_uint2(rescale4_by(w.x, f), rescale4_by(w.y, f));
                }
            }
        }
    }
    if (__builtin_expect(two_power(s), 1)) {
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tok + 4 * i;
            if (t >= m) continue;
            *reinterpret_cast<uint2*>(codes + (t0 + t) * 128 + c0) = encode8(x[i].a, inv);
            *reinterpret_cast<uint2*>(codes + (t0 + t) * 128 + c1) = encode8(x[i].b, inv);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = tok + 4 * i;
            if (t >= m) continue;
            auto by = [&](const uint4& v) {
                return make_uint2(encode2_by(v.x, s) | (encode2_by(v.y, s) << 16), encode2_by(v.z, s) | (encode2_by(v.w, s) << 16));
            };
            *reinterpret_cast<uint2*>(codes + (t0 + t) * 128 + c0) = by(x[i].a);
            *reinterpret_cast<uint2*>(codes + (t0 + t) * 128 + c1) = by(x[i].b);
        }
    }
    if (lane == 0) *scale_at = s;
}

// Two runs of one sequence in the call may meet in a region, whose warps do not know of each other: a
// block looks the rows over for that beside the others' work (a bit for each sequence, 2^15 sequences at a time).
__device__ __forceinline__ void check_runs(const AppendParams& p) {
    __shared__ uint32_t seen[kSeenWords];
    for (int64_t base = 0; base < p.B; base += kSeenWords * 32) {
        const int here = (int)min((int64_t)kSeenWords * 32, p.B - base);
        for (int i = threadIdx.x; i < (here + 31) / 32; i += kAppendThreads) seen[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int n = threadIdx.x; n < p.N; n += kAppendThreads) {
            const int b = p.row_seq[n], before = n > 0 ? p.row_seq[n - 1] : -1;
            const int64_t i = b - base;
            if (b == before || i < 0 || i >= here) continue;
            const uint32_t bit = 1u << (i & 31);
            if (atomicOr(&seen[i >> 5], bit) & bit) raise_status(p.status, kDevRange);
        }
        __syncthreads();
    }
}

template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (E4M3)
        if (blockIdx.x < p.check_blocks) return check_runs(p);
    const int lane = threadIdx.x & 31;
    const uint32_t id = (blockIdx.x - (E4M3 ? p.check_blocks : 0u)) * kAppendWarps + (threadIdx.x >> 5);
    if (!E4M3 || id >= p.region_warps) {
        append_row<E4M3>(p, E4M3 ? id - p.region_warps : id, lane);
        return;
    }
    // lane i: row n0 - 1 + i; lanes 1 .. rows_per_warp may lead a region
    const uint32_t u = id % (2 * p.G);
    const int n0 = (int)(id / (2 * p.G)) * p.rows_per_warp, rn = n0 - 1 + lane;
    int rb = -1, rp = -1;
    if (lane < 16 + 1 && rn >= 0 && rn < p.N) {
        rb = p.row_seq[rn];
        rp = p.row_pos[rn];
    }
    const int pb = __shfl_up_sync(0xffffffffu, rb, 1), pp = __shfl_up_sync(0xffffffffu, rp, 1);
    const bool mine = lane >= 1 && lane <= p.rows_per_warp;
    const bool in = rb >= 0 && rb < p.B && rp >= 0 && rp < p.pos_cap;
    const bool follows = pb == rb && pp == rp - 1, strays = pb == rb && !follows;  // strays: a sequence's rows out of order
    if (u == 0 && mine && ((!in && rb != -1) || (in && strays))) raise_status(p.status, kDevRange);
    uint32_t leads = __ballot_sync(0xffffffffu, mine && in && !strays && (!follows || (rp & 7) == 0));
    const uint32_t goes_on = __ballot_sync(0xffffffffu, in && follows && (rp & 7) != 0);
    for (; leads; leads &= leads - 1) {
        const int l = __ffs(leads) - 1;
        const int m = __ffs(~(goes_on >> 1 >> l));  // 1 + the rows that follow in the region
        append_region(p, n0 - 1 + l, m, __shfl_sync(0xffffffffu, rb, l), __shfl_sync(0xffffffffu, rp, l), (int)(u >> 1),
                      u & 1, lane);
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams& params, bool e4m3, cudaStream_t stream, bool pdl) {
    AppendParams p = params;
    // Warps to a row's vectors: 4 when the rows fill the GPU (each then takes two or three vectors a
    // lane; 2,048 rows in bf16 10.7 us against 15.1 with 16), 16 for few rows, whose latency counts (one
    // row 2.1 us against 2.9 with 4).  Rows a region warp looks over for leaders: 8 in chunks, one of
    // which leads (4 x 1,021 rows 16.5 us against 26.8 with 1), one in decode batches, where every row
    // leads (16 rows 3.0 us against 13 with 8, 1,024 rows 9.6 against 17.3).
    p.row_shift = p.N >= 512 ? 2 : 4;
    p.rows_per_warp = p.N >= 512 && p.N >= 8 * (int64_t)p.B ? 8 : 1;
    p.region_warps = e4m3 ? (uint32_t)((p.N + p.rows_per_warp - 1) / p.rows_per_warp * 2 * p.G) : 0u;
    const uint32_t warps = p.region_warps + (e4m3 && p.q == nullptr ? 0u : (uint32_t)p.N << p.row_shift);
    cudaLaunchConfig_t cfg = {};
    p.check_blocks = e4m3 && p.N > 1 ? 1u : 0u;
    cfg.gridDim = dim3((warps + kAppendWarps - 1) / kAppendWarps + p.check_blocks);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return e4m3 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<true>, p) : cudaLaunchKernelEx(&cfg, kv_append_kernel<false>, p);
}

}  // namespace step5
