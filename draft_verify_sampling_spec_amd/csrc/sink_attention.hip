// sink_attention.hip -- attention of drafted blocks under a sliding window in front
// of which the first tokens stay visible: entry points. The kernels and their
// notes are in attend_kernel.h; the tiles that hold sinks are read like the
// window's, so a call costs what one over sinks + window tokens does: 32 single
// tokens of 64 heads of 64 under a window of 128 with 4 sinks 7.9 us, 128 blocks of
// 3..9 rows x 4 heads under 2,048 with 64 sinks 96 (8 kv heads of 128, 3.2 TB/s), 4 blocks
// of 5 under 32,768 with 1,000 sinks 40 (3.7).
#include "attend_kernel.h"

// Without a window, or without sinks, the call is spec_verify_attention's.
extern "C" size_t spec_verify_attention_sinks_workspace_bytes(int B, int K, int q_heads,
                                                              int kv_heads, int head_dim,
                                                              int page_size, int max_pages,
                                                              int window, int sinks) {
    if (B < 1 || sinks < 0 || !shape_ok(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window)) {
        return 0;
    }
    return workspace_of(plan_of(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window,
                                window > 0 ? sinks : 0), head_dim);
}

extern "C" int spec_verify_attention_sinks(const void* queries, int64_t query_stride,
                                           const void* cache, const int32_t* page_table,
                                           const int32_t* ctx_lens, const int32_t* budgets, int B,
                                           int K, int q_heads, int kv_heads, int head_dim,
                                           int page_size, int max_pages, int num_pages, float scale,
                                           int window, int sinks, void* out, int32_t* out_status,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    if (sinks < 0) return SV_ERR_ARG;
    if (window <= 0 || sinks == 0) {
        return spec_verify_attention(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K,
                                     q_heads, kv_heads, head_dim, page_size, max_pages, num_pages, scale,
                                     window, out, out_status, workspace, workspace_bytes, stream);
    }
    return attend<kSinks>(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K, q_heads,
                          kv_heads, head_dim, page_size, max_pages, num_pages, scale, window, sinks, out,
                          out_status, workspace, workspace_bytes, stream);
}
