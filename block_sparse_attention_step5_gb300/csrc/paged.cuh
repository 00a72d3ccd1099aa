// paged.cuh -- the paged KV cache: its addressing, and the parameter blocks and launchers
// of the kernels that write and read it.
#pragma once

#include <cuda.h>

#include "kernels.cuh"

namespace step5 {

// A pool of pages [num_pages][G][page_tokens][128] and the block table [B][table_len] that
// lists each sequence's pages (null: sequence b owns page b).
struct PageMap {
    const int32_t* table;
    int num_pages, page_tokens, table_len;
};

// The pool row (token row of 128 values; its scale is that of row / 8) of token `tok` of
// sequence b in group g, or -1 where the table names no page.
__device__ __forceinline__ int64_t page_row(const PageMap& m, int G, int b, int g, int tok) {
    const int slot = tok / m.page_tokens;
    if (slot >= m.table_len) return -1;
    const int page = m.table ? m.table[(int64_t)b * m.table_len + slot] : b;
    if (page < 0 || page >= m.num_pages) return -1;
    return ((int64_t)page * G + g) * m.page_tokens + (tok - slot * m.page_tokens);
}

struct AppendParams {
    const uint16_t* q;   // [N][Hq][128], rows q_stride apart, or null
    const uint16_t* k;   // [N][G][128]
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;  // elements
    const int32_t* row_seq;
    const int32_t* row_pos;
    const uint16_t* cos;  // [pos_cap][rot / 2] or null
    const uint16_t* sin;
    uint16_t* q_out;      // [N][Hq][128]
    void* k_pages;
    void* v_pages;
    float* k_scales;      // e4m3 pages: [num_pages][G][page_tokens / 8]
    float* v_scales;
    PageMap pages;
    uint32_t* status;
    int N, B, G, Hq, rot, pos_cap;
    int row_shift, rows_per_warp;  // the launch's split of the work: N <= 2^24 keeps it in 32 bits
    uint32_t region_warps, check_blocks;
};
cudaError_t launch_append(const AppendParams& p, bool e4m3, cudaStream_t stream, bool pdl);

struct PagedAttnParams {
    const uint16_t* q;       // [N][Hq][128]
    const uint8_t* k_pages;
    const uint8_t* v_pages;
    const float* k_scales;
    const float* v_scales;
    PageMap pages;
    const int32_t* row_seq;
    const int32_t* row_pos;
    const int32_t* sel_ids;    // [N][G][top_k], or null: every token of the window
    const int32_t* sel_count;  // [N][G]
    const uint16_t* gate;      // [N][Hq] bf16 logits or null
    uint16_t* out;             // [N][Hq][128]
    uint32_t* status;
    int4* shared_items;        // workspace: [kPagedMaxCtas], items that CTAs share: (n, g, first CTA, last CTA or -1)
    float* states;             // workspace: partial states of items that CTAs share
    int N, B, G, Hq, top_k, window;
    int box_regions;           // regions of one TMA box (a power of two <= 16 that divides a page's)
    float scale_log2;          // softmax_scale * log2(e)
};
constexpr int kPagedMaxCtas = 480;           // of one launch
constexpr size_t kPagedItemBytes = 16 * 512;
constexpr int kChunkMaxCtas = 160;           // of a launch of the kernel for several rows a sequence
// two states a CTA: of up to 16 heads each, or of 256 head rows
constexpr size_t kPagedStateFloats = (size_t)kChunkMaxCtas * 2 * 256 * 130;
static_assert((size_t)kPagedMaxCtas * 2 * 16 * 130 <= kPagedStateFloats, "workspace");
constexpr size_t kPagedWorkspaceBytes = kPagedItemBytes + kPagedStateFloats * 4;
// kmap, vmap: the pools as [rows][128] bytes, boxes of 8 * box_regions rows, 128-byte swizzle
cudaError_t launch_paged_attention(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   int num_sms, cudaStream_t stream, bool pdl);
// The same for launches whose sequences have several rows (no picks).
cudaError_t launch_paged_chunk(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int num_sms,
                               cudaStream_t stream, bool pdl);

// A scale that can be used: positive and at most 2^126 (so that the power of two above it is finite).
__device__ __forceinline__ bool scale_ok(float s) { return s > 0.0f && s <= 8.507059173e37f; }

}  // namespace step5
