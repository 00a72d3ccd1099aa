// paged_attention.cu -- attention over the e4m3 paged cache: every token of a causal window,
// or the picked regions plus the row's own.
//
//   s_t = softmax_scale (q . code_t) kscale(region of t),  out = sum_t p_t vscale code_t,  p = softmax(s)
//
// One block per (row, KV group); each warp takes every fourth region, its lanes four dims
// each, with one pass over the keys (running maximum and sum per head), and the warps' states
// meet in shared memory.
#include "paged.cuh"

namespace step5 {

namespace {

constexpr int kPgWarps = 4;

template <int HQ>
__global__ void __launch_bounds__(kPgWarps * 32) paged_attn_kernel(PagedAttnParams p) {
    __shared__ float sm[kPgWarps][HQ], sl[kPgWarps][HQ], so[kPgWarps][HQ][128];
    pdl_wait();
    pdl_launch_dependents();
    const int n = blockIdx.x, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t h0 = (int64_t)n * p.Hq + (int64_t)g * HQ;
    const int b = p.row_seq[n], pos = p.row_pos[n];
    if (b == -1) return;
    if (b < 0 || b >= p.B || pos < 0 || pos / p.pages.page_tokens >= p.pages.table_len) {
        if (threadIdx.x == 0) raise_status(p.status, kDevRange);
        for (int i = threadIdx.x; i < HQ * 128; i += kPgWarps * 32) p.out[h0 * 128 + i] = 0;
        return;
    }
    const int own = pos >> 3;
    const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    int cnt = own - (lo >> 3);  // entries before the own region
    if (p.sel_ids) {
        cnt = p.sel_count[(int64_t)n * p.G + g];
        if (cnt < 0 || cnt > p.top_k) {
            if (threadIdx.x == 0) raise_status(p.status, kDevRange);
            cnt = cnt < 0 ? 0 : p.top_k;
        }
    }
    float q[HQ][4], m[HQ], l[HQ], o[HQ][4];
#pragma unroll
    for (int h = 0; h < HQ; ++h) {
        const uint2 v = *reinterpret_cast<const uint2*>(p.q + (h0 + h) * 128 + lane * 4);
        q[h][0] = bf16_lo(v.x), q[h][1] = bf16_hi(v.x), q[h][2] = bf16_lo(v.y), q[h][3] = bf16_hi(v.y);
        m[h] = -INFINITY, l[h] = 0.0f;
        o[h][0] = o[h][1] = o[h][2] = o[h][3] = 0.0f;
    }
    for (int e = warp; e <= cnt; e += kPgWarps) {
        int r = own;
        if (e < cnt) r = p.sel_ids ? p.sel_ids[((int64_t)n * p.G + g) * p.top_k + e] : (lo >> 3) + e;
        if (r < 0 || r > own || (p.sel_ids && e < cnt && r == own)) {
            if (lane == 0) raise_status(p.status, kDevRange);
            continue;
        }
        const int64_t row = page_row(p.pages, p.G, b, g, r * 8);
        const float ks = row < 0 ? 0.0f : p.k_scales[row >> 3], vs = row < 0 ? 0.0f : p.v_scales[row >> 3];
        if (!(ks > 0.0f) || !(vs > 0.0f) || ks > 3.0e38f || vs > 3.0e38f) {
            if (lane == 0) raise_status(p.status, kDevRange);
            continue;
        }
        for (int t = 0; t < 8; ++t) {
            const int tok = r * 8 + t;
            if (tok < lo || tok > pos) continue;
            const uint32_t kc = *reinterpret_cast<const uint32_t*>(p.k_pages + (row + t) * 128 + lane * 4);
            const uint32_t vc = *reinterpret_cast<const uint32_t*>(p.v_pages + (row + t) * 128 + lane * 4);
            const float2 k0 = e4m3x2_to_f32x2((uint16_t)kc), k1 = e4m3x2_to_f32x2((uint16_t)(kc >> 16));
            const float2 v0 = e4m3x2_to_f32x2((uint16_t)vc), v1 = e4m3x2_to_f32x2((uint16_t)(vc >> 16));
#pragma unroll
            for (int h = 0; h < HQ; ++h) {
                float s = q[h][0] * k0.x + q[h][1] * k0.y + q[h][2] * k1.x + q[h][3] * k1.y;
#pragma unroll
                for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                s *= ks * p.scale_log2;
                const float mn = fmaxf(m[h], s);
                const float a = exp2f(m[h] - mn), w = exp2f(s - mn);
                m[h] = mn;
                l[h] = l[h] * a + w;
                const float wv = w * vs;
                o[h][0] = o[h][0] * a + wv * v0.x;
                o[h][1] = o[h][1] * a + wv * v0.y;
                o[h][2] = o[h][2] * a + wv * v1.x;
                o[h][3] = o[h][3] * a + wv * v1.y;
            }
        }
    }
#pragma unroll
    for (int h = 0; h < HQ; ++h) {
        if (lane == 0) sm[warp][h] = m[h], sl[warp][h] = l[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) so[warp][h][lane * 4 + i] = o[h][i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < HQ * 128; i += kPgWarps * 32) {
        const int h = i >> 7, d = i & 127;
        float M = -INFINITY, L = 0.0f, O = 0.0f;
        for (int w = 0; w < kPgWarps; ++w) M = fmaxf(M, sm[w][h]);
        for (int w = 0; w < kPgWarps; ++w) {
            if (sm[w][h] == -INFINITY) continue;
            const float a = exp2f(sm[w][h] - M);
            L += a * sl[w][h];
            O += a * so[w][h][d];
        }
        float gf = 1.0f;
        if (p.gate) gf = 1.0f / (1.0f + expf(-bf16_to_f32(p.gate[h0 + h])));
        p.out[(h0 + h) * 128 + d] = f32_to_bf16_bits(L > 0.0f ? O / L * gf : (L == 0.0f ? 0.0f : L));
    }
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams& p, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.N, (unsigned)p.G);
    cfg.blockDim = dim3(kPgWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    switch (p.Hq / p.G) {
        case 4: return cudaLaunchKernelEx(&cfg, paged_attn_kernel<4>, p);
        case 8: return cudaLaunchKernelEx(&cfg, paged_attn_kernel<8>, p);
        case 16: return cudaLaunchKernelEx(&cfg, paged_attn_kernel<16>, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace step5
