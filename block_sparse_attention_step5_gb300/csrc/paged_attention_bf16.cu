// paged_attention_bf16.cu -- attention over the bf16 paged cache: every token of a causal window, or the picked
// regions plus the row's own.
//
//   s_t = softmax_scale (q . k_t),  p = softmax(s),  out = sum_t p_t v_t
//
// A block takes a (row, group): each of its warps every fourth region of the row's keys, four lanes to a token's
// scores, every lane four of the output's dims; running maxima and sums in fp32, the warps' states joined in
// shared memory.
#include "paged_device.cuh"

namespace step5 {

namespace {

constexpr int kWarps = 4;

template <int H>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_bf16_kernel(PagedAttnParams p) {
    __shared__ float sq[H][128], so[kWarps][H][128], sm[kWarps][H], sl[kWarps][H];
    const int n = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int b = p.row_seq[n], pos = p.row_pos[n];
    if (b == -1) return;
    const int64_t head0 = (int64_t)n * p.Hq + g * H;
    if (b < 0 || b >= p.B || pos < 0 || pos / p.pages.page_tokens >= p.pages.table_len) {
        if (tid == 0) raise_status(p.status, kDevRange);
        for (int i = tid; i < H * 128; i += kWarps * 32) p.out[head0 * 128 + i] = 0;
        return;
    }
    for (int i = tid; i < H * 128; i += kWarps * 32)
        sq[i >> 7][i & 127] = bf16_to_f32(p.q[n * p.q_stride + g * H * 128 + i]) * p.scale_log2;
    __syncthreads();
    const int own = pos >> 3;
    int lo = 0, r0 = 0, entries;
    const int32_t* ids = nullptr;
    if (p.sel_ids != nullptr) {
        const int64_t ng = (int64_t)n * p.G + g;
        const int c = p.sel_count[ng];
        if (tid == 0 && (c < 0 || c > p.top_k)) raise_status(p.status, kDevRange);
        entries = min(max(c, 0), p.top_k) + 1;
        ids = p.sel_ids + ng * p.top_k;
    } else {
        lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        r0 = lo >> 3;
        entries = own - r0 + 1;
    }
    const uint16_t *kp = reinterpret_cast<const uint16_t*>(p.k_pages), *vp = reinterpret_cast<const uint16_t*>(p.v_pages);
    float m[H], l[H], o[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h) m[h] = -INFINITY, l[h] = o[h][0] = o[h][1] = o[h][2] = o[h][3] = 0.0f;
    for (int e = warp; e < entries; e += kWarps) {
        const bool last = e == entries - 1;
        const int r = ids == nullptr ? r0 + e : last ? own : ids[e];
        int64_t row = -1;
        if (r >= 0 && (last ? r == own : r < own)) row = page_row(p.pages, p.G, b, g, r * 8);
        if (row < 0) {
            raise_status(p.status, kDevRange);
            continue;
        }
        const int t = lane >> 2, part = lane & 3, tok = r * 8 + t;
        const bool sees = tok >= lo && tok <= pos;
        float s[H];
#pragma unroll
        for (int h = 0; h < H; ++h) s[h] = 0.0f;
        for (int d = part * 32; d < part * 32 + 32; ++d) {
            const float k = bf16_to_f32(kp[(row + t) * 128 + d]);
#pragma unroll
            for (int h = 0; h < H; ++h) s[h] = fmaf(sq[h][d], k, s[h]);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
            if (!sees) s[h] = -INFINITY;
            float mx = s[h];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float nm = fmaxf(m[h], mx), base = nm == -INFINITY ? 0.0f : nm, a = exp2f(m[h] - base);
            m[h] = nm;
            s[h] = sees ? exp2f(s[h] - base) : 0.0f;
            l[h] *= a;
#pragma unroll
            for (int x = 0; x < 4; ++x) o[h][x] *= a;
        }
        for (int i = 0; i < 8; ++i) {
            if (!__shfl_sync(0xffffffffu, sees, i * 4)) continue;
            const uint2 v = *reinterpret_cast<const uint2*>(vp + (row + i) * 128 + lane * 4);
            const float f[4] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float w = __shfl_sync(0xffffffffu, s[h], i * 4);
                l[h] += w;
#pragma unroll
                for (int x = 0; x < 4; ++x) o[h][x] = fmaf(w, f[x], o[h][x]);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
        *reinterpret_cast<float4*>(&so[warp][h][lane * 4]) = make_float4(o[h][0], o[h][1], o[h][2], o[h][3]);
        if (lane == 0) sm[warp][h] = m[h], sl[warp][h] = l[h];
    }
    __syncthreads();
    for (int h = 0; h < H; ++h) {
        float M = -INFINITY, L = 0.0f, O = 0.0f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float a = sm[w][h] == -INFINITY ? 0.0f : exp2f(sm[w][h] - M);
            L += a * sl[w][h];
            O += a * so[w][h][tid];
        }
        O = L == 0.0f ? 0.0f : O / L;
        if (p.gate != nullptr && L != 0.0f) O *= 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[head0 + h])));
        p.out[(head0 + h) * 128 + tid] = f32_to_bf16_bits(O);
    }
}

}  // namespace

cudaError_t launch_paged_attention_bf16(const PagedAttnParams& p, int num_sms, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.N, (unsigned)p.G);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    switch (p.Hq / p.G) {
        case 4: return cudaLaunchKernelEx(&cfg, paged_attn_bf16_kernel<4>, p);
        case 8: return cudaLaunchKernelEx(&cfg, paged_attn_bf16_kernel<8>, p);
        case 16: return cudaLaunchKernelEx(&cfg, paged_attn_bf16_kernel<16>, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace step5
