// Entry points of the attention over paged rows: argument checks, workspace
// layout and the choice of passes.
#include <type_traits>

#include "attend_split.cuh"

namespace cpkv {
namespace {

constexpr int kFewSeqs = 16;

// What both entry points are told of rows, heads and results.
struct HeadArgs {
  int dtype, q_heads, kv_heads, head_dim;
};

int check_heads(const HeadArgs &a) {
  if (a.dtype != CPKV_BF16 && a.dtype != CPKV_FP16) return CPKV_ERR_ARG;
  if (a.kv_heads < 1 || a.q_heads < 1 || a.q_heads % a.kv_heads != 0) return CPKV_ERR_ARG;
  if (a.head_dim != 64 && a.head_dim != 128) return CPKV_ERR_LIMIT;
  if (a.q_heads > 4096) return CPKV_ERR_LIMIT;
  return CPKV_OK;
}

int check_rows(const HeadArgs &a, int64_t row_bytes, int64_t k_off, int64_t v_off) {
  const int64_t bytes = (int64_t)a.kv_heads * a.head_dim * 2;
  if (k_off < 0 || v_off < 0 || k_off % 16 != 0 || v_off % 16 != 0) return CPKV_ERR_ARG;
  if (k_off + bytes > row_bytes || v_off + bytes > row_bytes) return CPKV_ERR_ARG;
  return CPKV_OK;
}

int fill_io(AttendIo *io, const HeadArgs &a, const void *q, int64_t q_stride, void *out, int64_t out_stride, float *lse,
            float scale, int64_t k_off, int64_t v_off) {
  const int64_t width = (int64_t)a.q_heads * a.head_dim;
  if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out)) return CPKV_ERR_ARG;
  if (q_stride < width || out_stride < width || q_stride % 8 != 0 || out_stride % 8 != 0) return CPKV_ERR_ARG;
  if (!(scale > -INFINITY && scale < INFINITY)) return CPKV_ERR_ARG;
  io->q = static_cast<const char *>(q);
  io->out = static_cast<char *>(out);
  io->lse = lse;
  io->q_stride = q_stride * 2;
  io->out_stride = out_stride * 2;
  io->q_heads = a.q_heads;
  io->kv_heads = a.kv_heads;
  io->group = fast_div((uint32_t)(a.q_heads / a.kv_heads));
  io->scale_log2 = scale * kLog2e;
  io->k_off = k_off;
  io->v_off = v_off;
  return CPKV_OK;
}

int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

// Bounds of a split pass, from host lengths.
struct SplitBounds {
  int64_t tokens = 0, tiles_cap = 0, units = 0;
  int grid_cap = 1;

  void add(int64_t nq, int64_t max_kv, int group, int kv_heads, int window, int sinks) {
    int64_t tiles = ceil_div(max_kv, kSplitTile);
    if (window > 0) tiles = std::min<int64_t>(tiles, ceil_div((int64_t)sinks, kSplitTile) + ((int64_t)window + nq) / kSplitTile + 2);
    units += ceil_div(nq * group, kSplitRows) * kv_heads * tiles;
    tokens += nq;
  }
  int finish(int64_t count, int group) {
    tiles_cap = tokens * group / kSplitRows + count;
    if (units > INT32_MAX || tokens * group > INT32_MAX) return CPKV_ERR_LIMIT;
    grid_cap = (int)std::min<int64_t>(kSplitMaxGrid, units > 0 ? units : 1);
    return CPKV_OK;
  }
  int64_t slots(int kv_heads, bool direct) const { return 2 * (int64_t)grid_cap + (direct ? 0 : tiles_cap * kv_heads); }
  int64_t bytes(int64_t count, int kv_heads, int head_dim, bool direct) const {
    const int64_t n = slots(kv_heads, direct) * kSplitRows;
    return round_up((count + 1) * 4, 256) + round_up(n * 8, 256) + round_up(n * head_dim * 4, 256);
  }
  SplitSpace space(char *at, int64_t count, int kv_heads, bool direct) const {
    SplitSpace s;
    s.cum = reinterpret_cast<int32_t *>(at);
    at += round_up((count + 1) * 4, 256);
    s.ml = reinterpret_cast<float *>(at);
    at += round_up(slots(kv_heads, direct) * kSplitRows * 8, 256);
    s.o = reinterpret_cast<float *>(at);
    s.grid = grid_cap;
    return s;
  }
};

int window_bounds(SplitBounds *b, const HeadArgs &a, int B, const int32_t *h_q_lens, int64_t max_kv, int window,
                  int sinks) {
  for (int s = 0; s < B; ++s) {
    const int64_t nq = h_q_lens == nullptr ? 1 : h_q_lens[s];
    if (nq < 0) return CPKV_ERR_ARG;
    b->add(nq, max_kv, a.q_heads / a.kv_heads, a.kv_heads, window, sinks);
  }
  return b->finish(B, a.q_heads / a.kv_heads);
}

template <typename F>
int for_type_and_dim(const HeadArgs &a, F f) {
  if (a.dtype == CPKV_BF16) {
    return a.head_dim == 128 ? f(__nv_bfloat16(), std::integral_constant<int, 128>())
                             : f(__nv_bfloat16(), std::integral_constant<int, 64>());
  }
  return a.head_dim == 128 ? f(__half(), std::integral_constant<int, 128>())
                           : f(__half(), std::integral_constant<int, 64>());
}

template <typename T, int D, int N>
int split_pass(SplitParams<N> *p, const SplitBounds &b, cudaStream_t stream) {
  const int smem = SplitShape<D>::kSmem + (p->seqs.count + 1) * 4;
  auto kernel = attend_split_kernel<T, D, N>;
  const int rc = ensure_dynamic_smem((const void *)kernel, SplitShape<D>::kSmem + (CPKV_MAX_BATCH + 1) * 4);
  if (rc != CPKV_OK) return rc;
  p->space.grid = persistent_grid((const void *)kernel, kSplitWarps * 32, smem, 8, b.grid_cap);
  return launch_kernel(kernel, dim3(p->space.grid), dim3(kSplitWarps * 32), smem, false, stream, *p);
}

template <int N>
SplitSource<N> source_of(const SplitParams<N> &p) {
  SplitSource<N> s;
  s.seqs = p.seqs;
  s.space = p.space;
  s.tiles_cap = p.tiles_cap;
  s.direct = p.direct;
  return s;
}

template <typename T, int D, int N, int M>
int join_pass(const JoinParams<N, M> &p, cudaStream_t stream) {
  const int64_t blocks = ceil_div(p.rows, 4);
  if (blocks > INT32_MAX) return CPKV_ERR_LIMIT;
  return launch_kernel(attend_join_kernel<T, D, N, M>, dim3((unsigned)blocks), dim3(128), 0, false, stream, p);
}

template <int N>
int attend_window(const HeadArgs &heads, const Seqs<N> &seqs, const PagedPools &pools, const AttendIo &io,
                  const SplitBounds &bounds, char *workspace, cudaStream_t stream) {
  SplitParams<N> p = {};
  p.seqs = seqs;
  p.pools = pools;
  p.io = io;
  p.space = bounds.space(workspace, seqs.count, heads.kv_heads, true);
  p.tiles_cap = bounds.tiles_cap;
  p.direct = 1;
  return for_type_and_dim(heads, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    const int rc = split_pass<T, D, N>(&p, bounds, stream);
    if (rc != CPKV_OK) return rc;
    JoinParams<N, kFewSeqs> j = {};
    j.a = source_of(p);
    j.io = io;
    j.rows = bounds.tokens * heads.q_heads;
    return join_pass<T, D, N, kFewSeqs>(j, stream);
  });
}

template <int N>
int attend_shared(const HeadArgs &heads, const Seqs<N> &prefix, const Seqs<kFewSeqs> &suffix, const PagedPools &pools,
                  const AttendIo &io, const SplitBounds &pb, const SplitBounds &sb, char *workspace,
                  cudaStream_t stream) {
  SplitParams<N> pp = {};
  pp.seqs = prefix;
  pp.pools = pools;
  pp.io = io;
  pp.space = pb.space(workspace, prefix.count, heads.kv_heads, false);
  pp.tiles_cap = pb.tiles_cap;
  SplitParams<kFewSeqs> sp = {};
  sp.seqs = suffix;
  sp.pools = pools;
  sp.io = io;
  sp.space = sb.space(workspace + pb.bytes(prefix.count, heads.kv_heads, heads.head_dim, false), suffix.count,
                      heads.kv_heads, false);
  sp.tiles_cap = sb.tiles_cap;
  return for_type_and_dim(heads, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    int rc = split_pass<T, D, N>(&pp, pb, stream);
    if (rc != CPKV_OK) return rc;
    rc = split_pass<T, D, kFewSeqs>(&sp, sb, stream);
    if (rc != CPKV_OK) return rc;
    JoinParams<kFewSeqs, N> j = {};
    j.a = source_of(sp);
    j.b = source_of(pp);
    j.two_passes = 1;
    j.io = io;
    j.rows = sb.tokens * heads.q_heads;
    return join_pass<T, D, kFewSeqs, N>(j, stream);
  });
}

int shared_bounds(SplitBounds *prefix, SplitBounds *suffix, const HeadArgs &a, int B, int n_groups,
                  const int32_t *h_group_sizes, const int32_t *h_prefix_lens, int page_size, int64_t max_suffix) {
  const int group = a.q_heads / a.kv_heads;
  int64_t sum = 0, pages = 0;
  for (int g = 0; g < n_groups; ++g) {
    if (h_group_sizes[g] < 0 || h_prefix_lens[g] < 0) return CPKV_ERR_ARG;
    if (page_size > 0 && h_prefix_lens[g] % page_size != 0) return CPKV_ERR_UNALIGNED_PREFIX;
    prefix->add(h_group_sizes[g], h_prefix_lens[g], group, a.kv_heads, 0, 0);
    sum += h_group_sizes[g];
    if (page_size > 0) pages += h_prefix_lens[g] / page_size;
  }
  if (sum != B) return CPKV_ERR_ARG;
  if (pages > INT32_MAX) return CPKV_ERR_LIMIT;
  for (int b = 0; b < B; ++b) suffix->add(1, max_suffix, group, a.kv_heads, 0, 0);
  const int rc = prefix->finish(n_groups, group);
  return rc != CPKV_OK ? rc : suffix->finish(B, group);
}

}  // namespace
}  // namespace cpkv

using namespace cpkv;

extern "C" int cpkv_attend_window_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim,
                                                  const int32_t *h_q_lens, int64_t max_kv_len, int window, int sinks,
                                                  int64_t *h_bytes) {
  const HeadArgs heads = {CPKV_BF16, q_heads, kv_heads, head_dim};
  if (B < 0 || max_kv_len < 0 || window < 0 || sinks < 0 || h_bytes == nullptr) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || max_kv_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  SplitBounds b;
  rc = window_bounds(&b, heads, B, h_q_lens, max_kv_len, window, sinks);
  if (rc != CPKV_OK) return rc;
  *h_bytes = b.bytes(B, kv_heads, head_dim, true);
  return CPKV_OK;
}

extern "C" int cpkv_attend_window(int B, int page_size, int cp_size, int dtype, int q_heads, int kv_heads, int head_dim,
                                  int64_t row_bytes, int64_t key_offset, int64_t value_offset,
                                  const int32_t *h_q_lens, int64_t max_kv_len, const void *const *h_pools,
                                  const int64_t *h_pool_cap_pages, const int32_t *d_page_table, int64_t table_stride,
                                  const int32_t *d_kv_lens, const void *d_q, int64_t q_stride, float scale, int window,
                                  int sinks, void *d_out, int64_t out_stride, float *d_lse, void *d_workspace,
                                  int64_t workspace_bytes, int flags, int32_t *d_status, cpkv_stream_t stream) {
  const HeadArgs heads = {dtype, q_heads, kv_heads, head_dim};
  if (B < 0 || max_kv_len < 0 || window < 0 || sinks < 0 || (flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || max_kv_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  PagedPools pools = {};
  rc = paged_pools(&pools, page_size, cp_size, row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  rc = check_rows(heads, row_bytes, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (table_stride < 0 || max_kv_len > table_stride * page_size) return CPKV_ERR_CAPACITY;
  SplitBounds bounds;
  rc = window_bounds(&bounds, heads, B, h_q_lens, max_kv_len, window, sinks);
  if (rc != CPKV_OK) return rc;
  if (bounds.tokens == 0) return CPKV_OK;
  if (d_kv_lens == nullptr || d_status == nullptr || (max_kv_len > 0 && d_page_table == nullptr)) return CPKV_ERR_ARG;
  AttendIo io = {};
  rc = fill_io(&io, heads, d_q, q_stride, d_out, out_stride, d_lse, scale, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (d_workspace == nullptr || !aligned16(d_workspace)) return CPKV_ERR_ARG;
  if (workspace_bytes < bounds.bytes(B, kv_heads, head_dim, true)) return CPKV_ERR_CAPACITY;
  bool uniform = true;
  for (int b = 1; b < B && h_q_lens != nullptr; ++b) uniform &= h_q_lens[b] == h_q_lens[0];
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Seqs<N> s = {};
    s.kv_lens = d_kv_lens;
    s.table = d_page_table;
    s.stride = table_stride;
    s.status = d_status;
    s.count = B;
    s.kv_cap = (int)max_kv_len;
    s.causal = 1;
    s.window = window;
    s.sinks = sinks;
    if (uniform) {
      s.uniform_q = h_q_lens == nullptr ? 1 : h_q_lens[0];
    } else {
      for (int b = 0; b < B; ++b) s.cu_q[b + 1] = s.cu_q[b] + h_q_lens[b];
    }
    return attend_window<N>(heads, s, pools, io, bounds, static_cast<char *>(d_workspace), (cudaStream_t)stream);
  };
  if (uniform || B <= kFewSeqs) return go(std::integral_constant<int, kFewSeqs>());
  return go(std::integral_constant<int, CPKV_MAX_BATCH>());
}

extern "C" int cpkv_attend_shared_workspace_bytes(int B, int n_groups, int q_heads, int kv_heads, int head_dim,
                                                  const int32_t *h_group_sizes, const int32_t *h_prefix_lens,
                                                  int64_t max_suffix_len, int64_t *h_bytes) {
  const HeadArgs heads = {CPKV_BF16, q_heads, kv_heads, head_dim};
  if (B < 0 || n_groups < 0 || max_suffix_len < 0 || h_bytes == nullptr) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || n_groups > CPKV_MAX_BATCH || max_suffix_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  if (n_groups > 0 && (h_group_sizes == nullptr || h_prefix_lens == nullptr)) return CPKV_ERR_ARG;
  SplitBounds pb, sb;
  rc = shared_bounds(&pb, &sb, heads, B, n_groups, h_group_sizes, h_prefix_lens, 0, max_suffix_len);
  if (rc != CPKV_OK) return rc;
  *h_bytes = pb.bytes(n_groups, kv_heads, head_dim, false) + sb.bytes(B, kv_heads, head_dim, false);
  return CPKV_OK;
}

extern "C" int cpkv_attend_shared(int B, int n_groups, int page_size, int cp_size, int dtype, int q_heads, int kv_heads,
                                  int head_dim, int64_t row_bytes, int64_t key_offset, int64_t value_offset,
                                  const int32_t *h_group_sizes, const int32_t *h_prefix_lens, int64_t max_suffix_len,
                                  const void *const *h_pools, const int64_t *h_pool_cap_pages,
                                  const int32_t *d_prefix_pages, const int32_t *d_page_table, int64_t table_stride,
                                  const int32_t *d_suffix_lens, const void *d_q, int64_t q_stride, float scale,
                                  void *d_out, int64_t out_stride, float *d_lse, void *d_workspace,
                                  int64_t workspace_bytes, int flags, int32_t *d_status, cpkv_stream_t stream) {
  const HeadArgs heads = {dtype, q_heads, kv_heads, head_dim};
  if (B < 0 || n_groups < 0 || max_suffix_len < 0 || (flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || n_groups > CPKV_MAX_BATCH || max_suffix_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  PagedPools pools = {};
  rc = paged_pools(&pools, page_size, cp_size, row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  rc = check_rows(heads, row_bytes, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (n_groups > 0 && (h_group_sizes == nullptr || h_prefix_lens == nullptr)) return CPKV_ERR_ARG;
  if (table_stride < 0 || max_suffix_len > table_stride * page_size) return CPKV_ERR_CAPACITY;
  SplitBounds pb, sb;
  rc = shared_bounds(&pb, &sb, heads, B, n_groups, h_group_sizes, h_prefix_lens, page_size, max_suffix_len);
  if (rc != CPKV_OK) return rc;
  if (B == 0) return CPKV_OK;
  if (d_suffix_lens == nullptr || d_status == nullptr || (max_suffix_len > 0 && d_page_table == nullptr) ||
      (pb.units > 0 && d_prefix_pages == nullptr))
    return CPKV_ERR_ARG;
  AttendIo io = {};
  rc = fill_io(&io, heads, d_q, q_stride, d_out, out_stride, d_lse, scale, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (d_workspace == nullptr || !aligned16(d_workspace)) return CPKV_ERR_ARG;
  if (workspace_bytes < pb.bytes(n_groups, kv_heads, head_dim, false) + sb.bytes(B, kv_heads, head_dim, false))
    return CPKV_ERR_CAPACITY;
  Seqs<kFewSeqs> suffix = {};
  suffix.kv_lens = d_suffix_lens;
  suffix.table = d_page_table;
  suffix.stride = table_stride;
  suffix.status = d_status;
  suffix.count = B;
  suffix.uniform_q = 1;
  suffix.kv_cap = (int)max_suffix_len;
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Seqs<N> s = {};
    s.table = d_prefix_pages;
    s.stride = -1;
    s.status = d_status;
    s.count = n_groups;
    int pages = 0;
    for (int g = 0; g < n_groups; ++g) {
      s.cu_q[g + 1] = s.cu_q[g] + h_group_sizes[g];
      s.kv[g] = h_prefix_lens[g];
      s.page0[g] = pages;
      pages += h_prefix_lens[g] / page_size;
    }
    return attend_shared<N>(heads, s, suffix, pools, io, pb, sb, static_cast<char *>(d_workspace), (cudaStream_t)stream);
  };
  if (n_groups <= kFewSeqs) return go(std::integral_constant<int, kFewSeqs>());
  return go(std::integral_constant<int, CPKV_MAX_BATCH>());
}
