// Attention for trees of drafted tokens over a paged K/V cache: the C entry
// point.  The kernel is dsa_paged_attention's with a mask for the drafts' keys,
// in a translation unit of its own so that the two compile in parallel.
#include "dsa_attention.cuh"

extern "C" dsa_status dsa_tree_attention(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache,
    const void* v_cache, int64_t k_stride_page, int64_t k_stride_token, int64_t k_stride_head,
    int64_t v_stride_page, int64_t v_stride_token, int64_t v_stride_head, int64_t num_pages,
    int32_t page_size, const int32_t* block_table, int64_t bt_stride, const int32_t* query_start,
    const int32_t* context_lens, int32_t max_context,
    const uint32_t* tree_mask, int32_t mask_words, int64_t mask_stride, float scale,
    int32_t window, int32_t sinks,
    void* out, int64_t out_stride_t, int64_t out_stride_h, float* lse, int32_t T, int32_t B,
    int32_t H, int32_t Hkv, int32_t head_dim, int32_t dtype, uint32_t flags, void* workspace,
    size_t workspace_bytes, int32_t* err_flags, void* stream) {
  return attend<true>(q, q_stride_t, q_stride_h, k_cache, v_cache, k_stride_page,
      k_stride_token, k_stride_head, v_stride_page, v_stride_token, v_stride_head, num_pages,
      page_size, block_table, bt_stride, query_start, context_lens, max_context, tree_mask,
      mask_words, mask_stride, scale, window, sinks, out, out_stride_t, out_stride_h, lse, T, B,
      H, Hkv, head_dim, dtype, flags, workspace, workspace_bytes, err_flags, stream);
}
