// paged_api.cu -- the C ABI of the paged KV cache: host-side validation and launches.
// Declared in include/step5_sparse_attn.h.
#include "api.cuh"
#include "paged.cuh"

using namespace step5;

namespace {

step5_status check_pages(const step5_geometry* g, const step5_pages* pages, int32_t N, int32_t B,
                         const int32_t* block_table) {
    const step5_status s = check_geometry(g);
    if (s != STEP5_OK) return s;
    if (pages == nullptr || N <= 0 || B <= 0) return STEP5_ERR_INVALID_ARGUMENT;
    if (pages->num_pages <= 0 || pages->page_tokens <= 0 || pages->table_len <= 0) return STEP5_ERR_INVALID_ARGUMENT;
    if (pages->page_tokens % g->region_tokens) return STEP5_ERR_INVALID_ARGUMENT;
    // without a table a sequence is its page
    if (block_table == nullptr && (pages->table_len != 1 || pages->num_pages < B)) return STEP5_ERR_INVALID_ARGUMENT;
    if ((int64_t)pages->page_tokens * pages->table_len > INT32_MAX ||
        (int64_t)pages->num_pages * g->num_kv_groups * pages->page_tokens > INT32_MAX)
        return STEP5_ERR_INVALID_ARGUMENT;
    return STEP5_OK;
}

// A pool of e4m3 codes as [rows][128] bytes, boxes of 8 * box_regions rows, 128-byte swizzle.
bool encode_pool_map(CUtensorMap* map, const void* base, uint64_t rows, int box_regions) {
    auto enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {128, rows};
    cuuint64_t strides[1] = {128};
    cuuint32_t box[2] = {128, (cuuint32_t)(8 * box_regions)};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

step5_status append_impl(const step5_geometry* geom, const step5_pages* pages, int32_t N, int32_t B, int32_t rot_dims,
                         int32_t t_cap, const void* q_bf16_or_null, int64_t q_stride, const void* k_bf16,
                         int64_t k_stride, const void* v_bf16, int64_t v_stride, const int32_t* row_seq,
                         const int32_t* row_pos, const void* rope_cos_bf16, const void* rope_sin_bf16,
                         void* q_out_bf16_or_null, void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                         const int32_t* block_table, bool e4m3, step5_stream_t stream) {
    step5_status s = check_pages(geom, pages, N, B, block_table);
    if (s != STEP5_OK) return s;
    if (t_cap <= 0 || !k_bf16 || !v_bf16 || !row_seq || !row_pos || !k_pages || !v_pages) return STEP5_ERR_INVALID_ARGUMENT;
    if (e4m3 && (!k_scales || !v_scales)) return STEP5_ERR_INVALID_ARGUMENT;
    if ((q_bf16_or_null == nullptr) != (q_out_bf16_or_null == nullptr)) return STEP5_ERR_INVALID_ARGUMENT;
    if ((rope_cos_bf16 == nullptr) != (rope_sin_bf16 == nullptr)) return STEP5_ERR_INVALID_ARGUMENT;
    if (rot_dims < 0 || rot_dims > geom->head_dim || rot_dims % 16) return STEP5_ERR_UNSUPPORTED;
    if (N > 1 << 24) return STEP5_ERR_UNSUPPORTED;
    const int64_t G = geom->num_kv_groups, Hq = geom->num_q_heads, D = geom->head_dim;
    if (k_stride < G * D || v_stride < G * D || k_stride % 8 || v_stride % 8) return STEP5_ERR_INVALID_ARGUMENT;
    if (q_bf16_or_null && (q_stride < Hq * D || q_stride % 8)) return STEP5_ERR_INVALID_ARGUMENT;
    if (!aligned16(q_bf16_or_null) || !aligned16(q_out_bf16_or_null) || !aligned16(k_bf16) || !aligned16(v_bf16) ||
        !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(rope_cos_bf16) || !aligned16(rope_sin_bf16))
        return STEP5_ERR_INVALID_ARGUMENT;
    uint32_t* st = status_ptr();
    if (!st) return STEP5_ERR_CUDA;
    AppendParams p;
    p.q = static_cast<const uint16_t*>(q_bf16_or_null);
    p.k = static_cast<const uint16_t*>(k_bf16);
    p.v = static_cast<const uint16_t*>(v_bf16);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.row_seq = row_seq;
    p.row_pos = row_pos;
    p.cos = static_cast<const uint16_t*>(rope_cos_bf16);
    p.sin = static_cast<const uint16_t*>(rope_sin_bf16);
    p.q_out = static_cast<uint16_t*>(q_out_bf16_or_null);
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.pages = {block_table, pages->num_pages, pages->page_tokens, pages->table_len};
    p.status = st;
    p.N = N;
    p.B = B;
    p.G = geom->num_kv_groups;
    p.Hq = geom->num_q_heads;
    p.rot = rope_cos_bf16 ? rot_dims : 0;
    p.pos_cap = pages->page_tokens * pages->table_len;
    if (p.rot > 0 && t_cap < p.pos_cap) p.pos_cap = t_cap;
    return launch_append(p, e4m3, (cudaStream_t)stream, true) == cudaSuccess ? STEP5_OK : STEP5_ERR_CUDA;
}

step5_status attend_impl(const step5_geometry* geom, const step5_pages* pages, int32_t N, int32_t B, int32_t window,
                         const void* q_bf16, const uint8_t* k_pages, const uint8_t* v_pages, const float* k_scales,
                         const float* v_scales, const int32_t* block_table, const int32_t* row_seq,
                         const int32_t* row_pos, const int32_t* sel_ids, const int32_t* sel_count, const void* gate,
                         void* out_bf16, void* workspace, size_t workspace_bytes, step5_stream_t stream) {
    step5_status s = check_pages(geom, pages, N, B, block_table);
    if (s != STEP5_OK) return s;
    if (window < 0) return STEP5_ERR_INVALID_ARGUMENT;
    if (N > 65535) return STEP5_ERR_UNSUPPORTED;
    if (!q_bf16 || !k_pages || !v_pages || !k_scales || !v_scales || !row_seq || !row_pos || !out_bf16)
        return STEP5_ERR_INVALID_ARGUMENT;
    if (!aligned16(q_bf16) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out_bf16) || !aligned16(workspace))
        return STEP5_ERR_INVALID_ARGUMENT;
    if (workspace == nullptr || workspace_bytes < step5_paged_workspace_bytes(geom)) return STEP5_ERR_WORKSPACE;
    uint32_t* st = status_ptr();
    if (!st) return STEP5_ERR_CUDA;
    PagedAttnParams p;
    p.q = static_cast<const uint16_t*>(q_bf16);
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.pages = {block_table, pages->num_pages, pages->page_tokens, pages->table_len};
    p.row_seq = row_seq;
    p.row_pos = row_pos;
    p.sel_ids = sel_ids;
    p.sel_count = sel_count;
    p.gate = static_cast<const uint16_t*>(gate);
    p.out = static_cast<uint16_t*>(out_bf16);
    p.status = st;
    p.shared_items = static_cast<int4*>(workspace);
    p.states = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPagedItemBytes);
    p.N = N;
    p.B = B;
    p.G = geom->num_kv_groups;
    p.Hq = geom->num_q_heads;
    p.top_k = geom->top_k;
    p.window = window;
    p.scale_log2 = geom->softmax_scale * 1.4426950408889634f;
    // every token: the largest boxes that pages are made of; picks: one region each
    p.box_regions = 1;
    if (sel_ids == nullptr)
        while (p.box_regions < 16 && (pages->page_tokens / 8) % (2 * p.box_regions) == 0) p.box_regions *= 2;
    CUtensorMap kmap, vmap;
    const uint64_t rows = (uint64_t)pages->num_pages * geom->num_kv_groups * pages->page_tokens;
    if (!encode_pool_map(&kmap, k_pages, rows, p.box_regions) || !encode_pool_map(&vmap, v_pages, rows, p.box_regions))
        return STEP5_ERR_CUDA;
    // Rows of a sequence share its keys' tiles from 64 head rows a sequence and 128 head rows in all on.  With 8
    // heads a group, microseconds shared and alone: 4 rows of each of 8 sequences of 8,192 tokens 74 and 45, 8 rows of each
    // of 4 52 and 45, 8 of 16 111 and 140; one sequence's 8 rows 32 and 19 (behind 65,536 tokens 62 and 72), its 16 rows 32 and
    // 27 (63 and 144), its 32 rows 33 and 45.  With 16 heads, 16 rows of one 33 and 38, 8 of 4 49 and 59; with 4 heads, 32 of one 32 and
    // 42, 16 of 4 54 and 66.
    const int64_t head_rows = (int64_t)N * (geom->num_q_heads / geom->num_kv_groups);
    const bool chunk = sel_ids == nullptr && head_rows >= 64 * (int64_t)B && head_rows >= 128;
    const cudaError_t e = chunk ? launch_paged_chunk(p, kmap, vmap, num_sms(), (cudaStream_t)stream, true)
                                : launch_paged_attention(p, kmap, vmap, num_sms(), (cudaStream_t)stream, true);
    return e == cudaSuccess ? STEP5_OK : STEP5_ERR_CUDA;
}

}  // namespace

extern "C" {

step5_status step5_kv_append(const step5_geometry* geom, const step5_pages* pages, int32_t N, int32_t B,
                             int32_t rot_dims, int32_t t_cap, const void* q_bf16_or_null, int64_t q_stride,
                             const void* k_bf16, int64_t k_stride, const void* v_bf16, int64_t v_stride,
                             const int32_t* row_seq, const int32_t* row_pos, const void* rope_cos_bf16,
                             const void* rope_sin_bf16, void* q_out_bf16_or_null, void* k_pages_bf16,
                             void* v_pages_bf16, const int32_t* block_table_or_null, step5_stream_t stream) {
    return append_impl(geom, pages, N, B, rot_dims, t_cap, q_bf16_or_null, q_stride, k_bf16, k_stride, v_bf16, v_stride,
                       row_seq, row_pos, rope_cos_bf16, rope_sin_bf16, q_out_bf16_or_null, k_pages_bf16, v_pages_bf16,
                       nullptr, nullptr, block_table_or_null, false, stream);
}

step5_status step5_kv_append_e4m3(const step5_geometry* geom, const step5_pages* pages, int32_t N, int32_t B,
                                  int32_t rot_dims, int32_t t_cap, const void* q_bf16_or_null, int64_t q_stride,
                                  const void* k_bf16, int64_t k_stride, const void* v_bf16, int64_t v_stride,
                                  const int32_t* row_seq, const int32_t* row_pos, const void* rope_cos_bf16,
                                  const void* rope_sin_bf16, void* q_out_bf16_or_null, uint8_t* k_pages_e4m3,
                                  uint8_t* v_pages_e4m3, float* k_scales_f32, float* v_scales_f32,
                                  const int32_t* block_table_or_null, step5_stream_t stream) {
    return append_impl(geom, pages, N, B, rot_dims, t_cap, q_bf16_or_null, q_stride, k_bf16, k_stride, v_bf16, v_stride,
                       row_seq, row_pos, rope_cos_bf16, rope_sin_bf16, q_out_bf16_or_null, k_pages_e4m3, v_pages_e4m3,
                       k_scales_f32, v_scales_f32, block_table_or_null, true, stream);
}

size_t step5_paged_workspace_bytes(const step5_geometry* geom) {
    return check_geometry(geom) == STEP5_OK ? kPagedWorkspaceBytes : 0;
}

step5_status step5_paged_attn_e4m3(const step5_geometry* geom, const step5_pages* pages, int32_t N, int32_t B,
                                   int32_t window, const void* q_bf16, const uint8_t* k_pages_e4m3,
                                   const uint8_t* v_pages_e4m3, const float* k_scales_f32, const float* v_scales_f32,
                                   const int32_t* block_table_or_null, const int32_t* row_seq, const int32_t* row_pos,
                                   const void* gate_bf16_or_null, void* out_bf16, void* workspace,
                                   size_t workspace_bytes, step5_stream_t stream) {
    return attend_impl(geom, pages, N, B, window, q_bf16, k_pages_e4m3, v_pages_e4m3, k_scales_f32, v_scales_f32,
                       block_table_or_null, row_seq, row_pos, nullptr, nullptr, gate_bf16_or_null, out_bf16, workspace,
                       workspace_bytes, stream);
}

step5_status step5_sparse_attn_e4m3(const step5_geometry* geom, const step5_pages* pages, int32_t N, int32_t B,
                                    const void* q_bf16, const uint8_t* k_pages_e4m3, const uint8_t* v_pages_e4m3,
                                    const float* k_scales_f32, const float* v_scales_f32,
                                    const int32_t* block_table_or_null, const int32_t* row_seq, const int32_t* row_pos,
                                    const int32_t* sel_ids, const int32_t* sel_count, const void* gate_bf16_or_null,
                                    void* out_bf16, void* workspace, size_t workspace_bytes, step5_stream_t stream) {
    if (sel_ids == nullptr || sel_count == nullptr) return STEP5_ERR_INVALID_ARGUMENT;
    return attend_impl(geom, pages, N, B, 0, q_bf16, k_pages_e4m3, v_pages_e4m3, k_scales_f32, v_scales_f32,
                       block_table_or_null, row_seq, row_pos, sel_ids, sel_count, gate_bf16_or_null, out_bf16,
                       workspace, workspace_bytes, stream);
}

}  // extern "C"
