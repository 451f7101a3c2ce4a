// cpkv_read_quantised: rows of quantised pools, named by slot, back into 16 bits.
//
// x = e4m3 * scale, in 32 bits and rounded once: exact in bf16 for the scales that
// the append writes, but for multiples of less than 2^-133 and what reaches 2^128.  Two operations an element: bytes bound it, the rows read once
// and the results, twice their size, written once.
#include "quantised.cuh"
#include "tcgen05.cuh"

namespace cpkv {
namespace {

constexpr int kReadThreads = 256;

struct ReadParams {
  PagedPools pools;
  const int64_t *slots;
  char *k, *v;
  int32_t *status;
  int64_t k_stride, v_stride;  // bytes between rows
  int64_t k_off, v_off, ks_off, vs_off;
  int n_rows, keys_kept;
  int k_units, units, groups;  // units of 16 elements (8 of keys that are kept): of the keys, of a row; a thread's units are `groups` apart
  int wide;                    // results start on 32 bytes
  FastDiv threads;             // threads of a row: groups
  FastDiv key_units, value_units;  // units of a scale
};

// A thread takes kEach units of 16 elements of one row: their loads are in flight
// together, and so is the slot of the row that it works on next.  Units of 8 took half as
// many instructions again, which bound the call (88832 rows of 8 heads of 128: 101 us).
template <typename T, int kEach>
__global__ void __launch_bounds__(kReadThreads) read_quantised_kernel(const __grid_constant__ ReadParams p) {
  const int64_t total = (int64_t)p.n_rows * p.threads.d, step = (int64_t)gridDim.x * kReadThreads;
  auto row_of = [&](int64_t id) { return id < INT32_MAX ? div_by((int)id, p.threads) : (int)(id / p.threads.d); };
  int64_t id = (int64_t)blockIdx.x * kReadThreads + threadIdx.x;
  int64_t slot = 0;
  if (id < total) slot = p.slots[row_of(id)];
  for (; id < total; id += step) {
    const int n = row_of(id), first = (int)(id - (int64_t)n * p.threads.d);
    const int64_t next = id + step, mine = slot;
    if (next < total) slot = p.slots[row_of(next)];
    const char *row = nullptr;
    if (mine >= 0) {
      const int64_t page = mine < INT32_MAX ? div_by((int)mine, p.pools.page_size) : mine / p.pools.page_size.d;
      row = page <= INT32_MAX ? page_address(p.pools, (int)page) : nullptr;
      if (row != nullptr) {
        row += (mine - page * p.pools.page_size.d) * p.pools.row_bytes;
      } else if (first == 0) {
        raise_status(p.status, CPKV_STATUS_PAGE_OOB);
      }
    }
    uint4 x[kEach];
    float scale[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int u = first + e * p.groups;
      x[e] = make_uint4(0, 0, 0, 0);
      scale[e] = 0.f;
      if (row == nullptr || u >= p.units) continue;
      if (u < p.k_units && p.keys_kept) {
        x[e] = ld_stream16(row + p.k_off + u * 16);
        continue;
      }
      const bool key = u < p.k_units;
      const int w = key ? u : u - p.k_units;
      x[e] = ld_stream16(row + (key ? p.k_off : p.v_off) + w * 16);
      scale[e] = __ldg(reinterpret_cast<const float *>(row + (key ? p.ks_off : p.vs_off)) + div_by(w, key ? p.key_units : p.value_units));
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int u = first + e * p.groups;
      if (u >= p.units) continue;
      const bool key = u < p.k_units;
      if (key && p.keys_kept) {
        *reinterpret_cast<uint4 *>(p.k + n * p.k_stride + u * 16) = x[e];
        continue;
      }
      char *const to = key ? p.k + n * p.k_stride + u * 32 : p.v + n * p.v_stride + (u - p.k_units) * 32;
      const uint4 lo = read_back8<T>(make_uint2(x[e].x, x[e].y), scale[e]), hi = read_back8<T>(make_uint2(x[e].z, x[e].w), scale[e]);
      if (p.wide) {
        const uint32_t both[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        store32(to, both);
      } else {
        reinterpret_cast<uint4 *>(to)[0] = lo;
        reinterpret_cast<uint4 *>(to)[1] = hi;
      }
    }
  }
}

}  // namespace
}  // namespace cpkv

extern "C" int cpkv_read_quantised(int64_t n_rows, int page_size, int cp_size, int dtype, const cpkv_quantised_row *h_row,
                                   const void *const *h_pools, const int64_t *h_pool_cap_pages, const int64_t *d_slots,
                                   void *d_k, int64_t k_stride, void *d_v, int64_t v_stride, int flags, int32_t *d_status,
                                   cpkv_stream_t stream) {
  using namespace cpkv;
  if (n_rows < 0 || (dtype != CPKV_BF16 && dtype != CPKV_FP16) || (flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_quantised_row(h_row);
  if (rc != CPKV_OK) return rc;
  if (n_rows > INT32_MAX) return CPKV_ERR_LIMIT;
  const cpkv_quantised_row &row = *h_row;
  ReadParams p = {};
  rc = paged_pools(&p.pools, page_size, cp_size, row.row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  if (n_rows == 0 || (d_k == nullptr && d_v == nullptr)) return n_rows == 0 ? CPKV_OK : CPKV_ERR_ARG;
  if (d_slots == nullptr || d_status == nullptr || !aligned16(d_k) || !aligned16(d_v)) return CPKV_ERR_ARG;
  const int64_t k_width = (int64_t)row.kv_heads * row.key_dim, v_width = (int64_t)row.kv_heads * row.value_dim;
  if (d_k != nullptr && (k_stride < k_width || k_stride % 8 != 0)) return CPKV_ERR_ARG;
  if (d_v != nullptr && (v_stride < v_width || v_stride % 8 != 0)) return CPKV_ERR_ARG;
  p.slots = d_slots;
  p.k = static_cast<char *>(d_k);
  p.v = static_cast<char *>(d_v);
  p.status = d_status;
  p.k_stride = k_stride * 2;
  p.v_stride = v_stride * 2;
  p.k_off = row.key_offset;
  p.v_off = row.value_offset;
  p.ks_off = row.key_scale_offset;
  p.vs_off = row.value_scale_offset;
  p.n_rows = (int)n_rows;
  p.keys_kept = row.keep_keys != 0;
  p.k_units = d_k == nullptr ? 0 : (int)(k_width / (row.keep_keys ? 8 : 16));
  p.units = p.k_units + (d_v == nullptr ? 0 : (int)(v_width / 16));
  p.key_units = fast_div((uint32_t)std::max(row.key_dim / 16, 1));
  p.value_units = fast_div((uint32_t)value_group(row) / 16);
  p.wide = ((reinterpret_cast<uintptr_t>(d_k) | reinterpret_cast<uintptr_t>(d_v) | (uintptr_t)p.k_stride | (uintptr_t)p.v_stride) & 31) == 0;
  // Four units a thread once every SM has its 2048 threads so, one before.
  const int each = n_rows * p.units >= (int64_t)device_sm_count() * 4 * 2048 ? 4 : 1;
  p.groups = (int)ceil_div(p.units, each);
  p.threads = fast_div((uint32_t)p.groups);
  auto kernel = dtype == CPKV_BF16 ? (each == 4 ? read_quantised_kernel<__nv_bfloat16, 4> : read_quantised_kernel<__nv_bfloat16, 1>)
                                   : (each == 4 ? read_quantised_kernel<__half, 4> : read_quantised_kernel<__half, 1>);
  const int grid = persistent_grid((const void *)kernel, kReadThreads, 0, 8, ceil_div(n_rows * p.groups, kReadThreads));
  return launch_kernel(kernel, dim3(grid), dim3(kReadThreads), 0, false, (cudaStream_t)stream, p);
}
