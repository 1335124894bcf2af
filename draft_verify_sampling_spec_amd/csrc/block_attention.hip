// block_attention.hip -- attention of drafted blocks over the paged 4-bit cache,
// all of it or a sliding window: entry points. The kernels and their notes are in
// attend_kernel.h.
#include "attend_kernel.h"

extern "C" size_t spec_verify_attention_workspace_bytes(int B, int K, int q_heads, int kv_heads,
                                                        int head_dim, int page_size, int max_pages,
                                                        int window) {
    if (B < 1 || !shape_ok(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window)) {
        return 0;
    }
    return workspace_of(plan_of(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window), head_dim);
}

extern "C" int spec_verify_attention(const void* queries, int64_t query_stride, const void* cache,
                                     const int32_t* page_table, const int32_t* ctx_lens,
                                     const int32_t* budgets, int B, int K, int q_heads,
                                     int kv_heads, int head_dim, int page_size, int max_pages,
                                     int num_pages, float scale, int window, void* out,
                                     int32_t* out_status, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    return attend<kWindow>(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K, q_heads,
                           kv_heads, head_dim, page_size, max_pages, num_pages, scale, window, 0, out,
                           out_status, workspace, workspace_bytes, stream);
}
