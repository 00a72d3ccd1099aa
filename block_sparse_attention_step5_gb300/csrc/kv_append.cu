// kv_append.cu -- the rows' keys and values into the paged cache (bf16, or e4m3 with a scale
// for each region and KV group), with NEOX rotation of k (and of q) on the way.
//
// Rotation is the indexer's (x1 c - x2 s, x2 c + x1 s over pairs (i, i + rot / 2) from bf16
// cos/sin, the exact sum rounded once to bf16).  A head vector is 256 bytes: sixteen lanes
// take 16 bytes each, and since rot / 2 is a multiple of 8 a lane's eight partners lie in one
// other lane of the sixteen, so rotation costs four shuffles and two 16-byte table loads.
//
// In e4m3 a region's eight tokens share a scale, so the sixteen lanes of the first row that
// falls into a region (its leader: a row on a region's first token, or one that does not
// continue the row before) take all of the call's tokens of that region for one (group, k or v):
//   s = max(the scale held, if the region holds earlier tokens; the smallest power of two
//           >= max |x| / 448; 2^-126),      code = e4m3(x / s).
// A power of two divides exactly, costs an e4m3 value no precision (it has an exponent of its
// own), and makes the rescaling of tokens already held exact unless they leave the normal range.
// Those are requantised only when a new token raises the scale.
#include "paged.cuh"

namespace step5 {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kUnitsPerBlock = kAppendThreads / 16;

// Eight bf16 values (dims 8 lane .. 8 lane + 7 of a head vector held by 16 lanes), rotated.
// Every lane of the warp takes part in the shuffles.
__device__ __forceinline__ uint4 rotate8(uint4 x, const AppendParams& p, int pos, int l16, bool valid) {
    const int half8 = p.rot >> 4;  // lanes that hold the first elements of the pairs
    const bool first = l16 < half8, second = !first && l16 < 2 * half8;
    const int partner = first ? l16 + half8 : (second ? l16 - half8 : l16);
    uint4 y;
    y.x = __shfl_sync(0xffffffffu, x.x, partner, 16);
    y.y = __shfl_sync(0xffffffffu, x.y, partner, 16);
    y.z = __shfl_sync(0xffffffffu, x.z, partner, 16);
    y.w = __shfl_sync(0xffffffffu, x.w, partner, 16);
    if (!(first || second) || !valid) return x;
    const int64_t at = (int64_t)pos * (p.rot >> 1) + 8 * (first ? l16 : l16 - half8);
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(p.cos + at));
    const uint4 s = __ldg(reinterpret_cast<const uint4*>(p.sin + at));
    auto two = [&](uint32_t xv, uint32_t yv, uint32_t cv, uint32_t sv) {
        const uint32_t lo = neox_rotate(bf16_lo(xv), bf16_lo(yv), bf16_lo(cv), bf16_lo(sv), first);
        const uint32_t hi = neox_rotate(bf16_hi(xv), bf16_hi(yv), bf16_hi(cv), bf16_hi(sv), first);
        return lo | (hi << 16);
    };
    return make_uint4(two(x.x, y.x, c.x, s.x), two(x.y, y.y, c.y, s.y), two(x.z, y.z, c.z, s.z),
                      two(x.w, y.w, c.w, s.w));
}

// The largest finite |bf16| of eight, as bits (NaN left out, infinity taken as the largest finite value).
__device__ __forceinline__ uint32_t amax8(uint4 x) {
    uint32_t m = 0;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
        if (a <= 0x7f80u) m = max(m, a);
        if (b <= 0x7f80u) m = max(m, b);
    }
    return min(m, 0x7f7fu);
}

// The smallest power of two s >= 2^-126 with |x| <= 448 s = 1.75 * 2^8 s, x given as bf16 bits.
__device__ __forceinline__ float scale_for(uint32_t amax) {
    const int e = (int)(amax >> 7) - 8 + ((amax & 127u) > 96u ? 1 : 0);  // biased exponent of s
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ uint2 encode8(uint4 x, float inv) {
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

template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, l16 = lane & 15;
    const int nq = p.q ? p.Hq : 0, per = nq + 2 * p.G;
    const int64_t u = (int64_t)blockIdx.x * kUnitsPerBlock + (threadIdx.x >> 4);
    const int64_t n64 = u / per;
    const int n = (int)n64, j = (int)(u - n64 * per);
    const bool have = n64 < p.N;
    int b = -1, pos = 0;
    if (have) {
        b = p.row_seq[n];
        pos = p.row_pos[n];
    }
    bool ok = have && b >= 0 && b < p.B && pos >= 0 && pos < p.pos_cap;
    if (have && !ok && b != -1 && j == 0 && l16 == 0) raise_status(p.status, kDevRange);
    const bool is_q = j < nq;
    const int g = is_q ? 0 : (j - nq) % p.G;
    const bool is_v = !is_q && j - nq >= p.G;

    if (!E4M3) {
        int64_t row = -1;
        const uint16_t* src = nullptr;
        uint16_t* dst = nullptr;
        if (ok) {
            if (is_q) {
                src = p.q + n * p.q_stride + (int64_t)j * 128;
                dst = p.q_out + ((int64_t)n * p.Hq + j) * 128;
            } else {
                row = page_row(p.pages, p.G, b, g, pos);
                if (row < 0) {
                    if (l16 == 0) raise_status(p.status, kDevRange);
                } else {
                    src = (is_v ? p.v + n * p.v_stride : p.k + n * p.k_stride) + (int64_t)g * 128;
                    dst = static_cast<uint16_t*>(is_v ? p.v_pages : p.k_pages) + row * 128;
                }
            }
        }
        uint4 x = make_uint4(0, 0, 0, 0);
        if (src) x = *reinterpret_cast<const uint4*>(src + l16 * 8);
        x = rotate8(x, p, pos, l16, src != nullptr && !is_v && p.rot > 0);
        if (dst) *reinterpret_cast<uint4*>(dst + l16 * 8) = x;
        return;
    }

    // rows n .. n + 7 of the same sequence, one to a lane: how many continue this row inside its region
    const int t0 = pos & 7;
    int cnt = 0;
    bool leads = false;
    {
        bool next = false;
        if (ok && !is_q && l16 > 0 && l16 < 8 - t0 && n + l16 < p.N)
            next = p.row_seq[n + l16] == b && p.row_pos[n + l16] == pos + l16 && pos + l16 < p.pos_cap;
        const uint32_t bits = (__ballot_sync(0xffffffffu, next) >> (lane & 16)) & 0xffffu;
        cnt = __ffs(~(bits >> 1));  // 1 + the run of following rows
    }
    int64_t row = -1;
    if (ok && !is_q) {
        const bool same = n > 0 && p.row_seq[n - 1] == b;
        const int before = same ? p.row_pos[n - 1] : -1;
        if (same && before != pos - 1) {  // a sequence's rows out of order
            if (l16 == 0) raise_status(p.status, kDevRange);
        } else {
            leads = !same || t0 == 0;
        }
        if (leads) {
            row = page_row(p.pages, p.G, b, g, pos);
            if (row < 0) {
                if (l16 == 0) raise_status(p.status, kDevRange);
                leads = false;
            }
        }
    }
    if (!leads) cnt = 0;
    if (ok && is_q) cnt = 1;
    const uint16_t* src = nullptr;
    int64_t stride = 0;
    if (is_q) {
        src = p.q + n * p.q_stride + (int64_t)j * 128;
    } else {
        stride = is_v ? p.v_stride : p.k_stride;
        src = (is_v ? p.v : p.k) + n * stride + (int64_t)g * 128;
    }
    const int most = __reduce_max_sync(0xffffffffu, cnt);  // the warp's two units take the same steps
    uint4 x[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
        x[t] = t < cnt ? *reinterpret_cast<const uint4*>(src + t * stride + l16 * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t < most) x[t] = rotate8(x[t], p, pos + t, l16, t < cnt && !is_v && p.rot > 0);
    // the scale held, read and written by the unit's first lane alone
    float* scale_at = leads ? (is_v ? p.v_scales : p.k_scales) + (row >> 3) : nullptr;
    float held = 1.0f;
    if (leads && t0 > 0 && l16 == 0) held = *scale_at;
    held = __shfl_sync(0xffffffffu, held, 0, 16);
    uint32_t amax = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) amax = max(amax, amax8(x[t]));
#pragma unroll
    for (int d = 8; d; d >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (cnt == 0) return;
    if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + ((int64_t)n * p.Hq + j) * 128 + l16 * 8) = x[0];
        return;
    }
    uint8_t* codes = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + (row - t0) * 128 + l16 * 8;
    float s = scale_for(amax);
    if (t0 > 0) {
        if (!scale_ok(held)) {
            if (l16 == 0) raise_status(p.status, kDevRange);
        } else if (held >= s) {
            s = held;
        } else {
            const float f = held / s;
            for (int t = 0; t < t0; ++t) {
                uint2* at = reinterpret_cast<uint2*>(codes + t * 128);
                const uint2 c = *at;
                *at = make_uint2(rescale4(c.x, f), rescale4(c.y, f));
            }
        }
    }
    const float inv = 1.0f / s;
#pragma unroll
    for (int t = 0; t < 8; ++t)
        if (t < cnt) *reinterpret_cast<uint2*>(codes + (t0 + t) * 128) = encode8(x[t], inv);
    if (l16 == 0) *scale_at = s;
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, bool e4m3, cudaStream_t stream, bool pdl) {
    const int64_t units = (int64_t)p.N * ((p.q ? p.Hq : 0) + 2 * p.G);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((units + kUnitsPerBlock - 1) / kUnitsPerBlock));
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
