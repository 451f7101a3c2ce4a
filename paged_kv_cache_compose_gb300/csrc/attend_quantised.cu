// Entry points of the attention over quantised rows.
#include "attend_host.cuh"

using namespace cpkv;

extern "C" int cpkv_attend_window_quantised_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim,
                                                            const int32_t *h_q_lens, int64_t max_kv_len, int window,
                                                            int sinks, int64_t *h_bytes) {
  return window_bytes(true, HeadArgs{CPKV_BF16, q_heads, kv_heads, head_dim}, B, h_q_lens, max_kv_len, window, sinks, h_bytes);
}

extern "C" int cpkv_attend_window_quantised(int B, int page_size, int cp_size, int dtype, int q_heads,
                                            const cpkv_quantised_row *h_row, const int32_t *h_q_lens, int64_t max_kv_len,
                                            const void *const *h_pools, const int64_t *h_pool_cap_pages,
                                            const int32_t *d_page_table, int64_t table_stride, const int32_t *d_kv_lens,
                                            int64_t num_tokens, const void *d_q, int64_t q_stride, float scale, int window,
                                            int sinks, void *d_out, int64_t out_stride, float *d_lse, void *d_workspace,
                                            int64_t workspace_bytes, int flags, int32_t *d_status, cpkv_stream_t stream) {
  HeadArgs heads;
  RowArgs rows = {page_size, cp_size, 0, 0, 0, nullptr, h_pools, h_pool_cap_pages, flags};
  const int rc = quantised_rows(&heads, &rows, dtype, q_heads, h_row);
  if (rc != CPKV_OK) return rc;
  const WindowCall call = {B, h_q_lens, max_kv_len, d_page_table, table_stride, d_kv_lens, num_tokens, window, sinks};
  const ResultArgs results = {d_q, q_stride, scale, d_out, out_stride, d_lse, d_workspace, workspace_bytes, d_status, (cudaStream_t)stream};
  return window_call<true>(heads, rows, call, results);
}

extern "C" int cpkv_attend_shared_quantised_workspace_bytes(int B, int n_groups, int q_heads, int kv_heads, int head_dim,
                                                            const int32_t *h_group_sizes, const int32_t *h_prefix_lens,
                                                            int64_t max_suffix_len, int64_t *h_bytes) {
  return shared_bytes(true, HeadArgs{CPKV_BF16, q_heads, kv_heads, head_dim}, B, n_groups, h_group_sizes, h_prefix_lens, max_suffix_len,
                      h_bytes);
}

extern "C" int cpkv_attend_shared_quantised(int B, int n_groups, int page_size, int cp_size, int dtype, int q_heads,
                                            const cpkv_quantised_row *h_row, const int32_t *h_group_sizes,
                                            const int32_t *h_prefix_lens, int64_t max_suffix_len,
                                            const void *const *h_pools, const int64_t *h_pool_cap_pages,
                                            const int32_t *d_prefix_pages, int64_t num_prefix_pages,
                                            const int32_t *d_page_table, int64_t table_stride,
                                            const int32_t *d_suffix_lens, const void *d_q, int64_t q_stride, float scale,
                                            void *d_out, int64_t out_stride, float *d_lse, void *d_workspace,
                                            int64_t workspace_bytes, int flags, int32_t *d_status, cpkv_stream_t stream) {
  HeadArgs heads;
  RowArgs rows = {page_size, cp_size, 0, 0, 0, nullptr, h_pools, h_pool_cap_pages, flags};
  const int rc = quantised_rows(&heads, &rows, dtype, q_heads, h_row);
  if (rc != CPKV_OK) return rc;
  const SharedCall call = {B, n_groups, h_group_sizes, h_prefix_lens, max_suffix_len, d_prefix_pages, num_prefix_pages, d_page_table,
                           table_stride, d_suffix_lens};
  const ResultArgs results = {d_q, q_stride, scale, d_out, out_stride, d_lse, d_workspace, workspace_bytes, d_status, (cudaStream_t)stream};
  return shared_call<true>(heads, rows, call, results);
}

extern "C" int cpkv_selftest_attend_quantised_timeout(int head_dim, int n_tokens, int n_pages, const void *d_rows,
                                                      const int32_t *d_page_table, const int32_t *d_kv_len, const void *d_q,
                                                      void *d_out, int64_t wait_ns, int32_t *d_status, cpkv_stream_t stream) {
  constexpr int kPage = 64;
  if (n_tokens <= kSplitRows || n_pages < 1 || n_pages > (1 << 20) || wait_ns < 0) return CPKV_ERR_ARG;
  if (d_rows == nullptr || d_page_table == nullptr || d_kv_len == nullptr || d_status == nullptr) return CPKV_ERR_ARG;
  const cpkv_quantised_row row = {2 * (int64_t)head_dim + 16, 0, head_dim, 2 * (int64_t)head_dim, 2 * (int64_t)head_dim + 4, 1, head_dim, head_dim, 0};
  const int64_t cap = n_pages;
  HeadArgs heads;
  RowArgs rows = {kPage, 1, 0, 0, 0, nullptr, &d_rows, &cap, CPKV_DENSE_PAGES};
  const int rc = quantised_rows(&heads, &rows, CPKV_BF16, 1, &row);
  if (rc != CPKV_OK) return rc;
  const ResultArgs results = {d_q, head_dim, 0.125f, d_out, head_dim, nullptr, nullptr, 0, d_status, (cudaStream_t)stream};
  return selftest_call<true>(heads, rows, n_tokens, n_pages, d_page_table, d_kv_len, results, wait_ns);
}
