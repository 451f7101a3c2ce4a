// cpkv_append_rotary: new keys and values into the paged pools, keys (and
// queries beside them) rotated by their positions on the way.
//
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a
//
// for each pair (x1, x2) of frequency i, with cos a and sin a of row
// pos[axis(i)] of the caller's table.  Three multiplications and additions per
// element, so bytes bound it (and, for a few tokens, the launch): every row is
// read once and written once, products are held in 32 bits and rounded once.
#include "append.cuh"

namespace cpkv {
namespace {

// A thread owns one unit of a token and works through kEach heads with it: half
// / 8 units of a head are 16 rotated elements (8 frequencies, two 16-byte
// vectors), the others 16 plain ones (or the last 8).  The angles are looked up
// once for the kEach heads, whose loads are all in flight together.  Neighbouring
// threads hold a head's neighbouring units, so warps read and write whole heads.
// The threads after those copy kEach 16-byte chunks of the values each.
template <typename T, bool kPairs, bool kAxes, int kEach>
CPKV_DEV void do_work(const AppendParams &p, const Work<kAxes> &w) {
  const int n = w.n, u = w.u;
  const bool ok = w.positions_ok(p);
  if (u >= p.rotated) {  // values
    const char *src = p.v + n * p.v_stride;
    const int first = u - p.rotated;
    uint4 x[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int c = first + e * p.value_groups;
      if (c < p.value_chunks) x[e] = ld_stream16(src + c * 16);
    }
    char *const row = ok ? slot_row(p, w.slot, false) : nullptr;
    if (row == nullptr) return;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int c = first + e * p.value_groups;
      if (c < p.value_chunks) *reinterpret_cast<uint4 *>(row + p.v_off + c * 16) = x[e];
    }
    return;
  }

  const int first = div_by(u, p.head_units), unit = u - first * (int)p.head_units.d;
  const bool turns = unit * 8 < p.half;
  const int head_bytes = p.key_dim * 2;
  const int a0 = turns && !kPairs ? unit * 16 : unit * 32;  // plain units follow the rotated 2 half elements
  const int a1 = turns && !kPairs ? a0 + p.half * 2 : a0 + 16;
  const bool two = a1 < head_bytes;
  const char *const q = p.q + n * p.q_stride, *const k = p.k + n * p.k_stride;
  char *const q_out = p.q_out + n * p.q_out_stride;
  uint4 x0[kEach], x1[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int head = first + e * p.head_groups;
    if (head >= p.heads) continue;
    const char *src = head < p.q_heads ? q + head * head_bytes : k + (head - p.q_heads) * head_bytes;
    x0[e] = ld_stream16(src + a0);
    if (two) x1[e] = ld_stream16(src + a1);
  }
  float c[8], s[8];
  if (turns && ok) {
    angles4<kAxes>(p, w, unit * 8, c, s);
    angles4<kAxes>(p, w, unit * 8 + 4, c + 4, s + 4);
  }
  if (!ok && u == 0) raise_status(p.status, CPKV_STATUS_POS_OOB);
  char *const row = ok ? slot_row(p, w.slot, u == 0) : nullptr;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int head = first + e * p.head_groups;
    if (head >= p.heads) continue;
    char *dst;
    if (head < p.q_heads) {
      dst = q_out + head * head_bytes;
      if (!ok) x0[e] = x1[e] = make_uint4(0, 0, 0, 0);
    } else {
      if (row == nullptr) continue;
      dst = row + p.k_off + (head - p.q_heads) * head_bytes;
    }
    if (turns && ok) rotate_unit<T, kPairs>(x0[e], x1[e], c, s);
    *reinterpret_cast<uint4 *>(dst + a0) = x0[e];
    if (two) *reinterpret_cast<uint4 *>(dst + a1) = x1[e];
  }
}

// A grid that stays resident walks the units; a unit's token is looked up one step
// ahead.  Blocks of their own for every 128 units spent a seventh of their time on
// coming and going.
template <typename T, bool kPairs, bool kAxes, int kEach>
__global__ void __launch_bounds__(kAppendThreads) append_rotary_kernel(const __grid_constant__ AppendParams p) {
  const int64_t total = (int64_t)p.n_tokens * p.threads.d, step = (int64_t)gridDim.x * kAppendThreads;
  Work<kAxes> w = find_work<kAxes>(p, (int64_t)blockIdx.x * kAppendThreads + threadIdx.x, total);
  while (w.id < total) {
    const Work<kAxes> next = find_work<kAxes>(p, w.id + step, total);
    do_work<T, kPairs, kAxes, kEach>(p, w);
    w = next;
  }
}

template <typename T, int kEach>
auto append_kernel(bool pairs, bool axes) {
  if (pairs) return axes ? append_rotary_kernel<T, true, true, kEach> : append_rotary_kernel<T, true, false, kEach>;
  return axes ? append_rotary_kernel<T, false, true, kEach> : append_rotary_kernel<T, false, false, kEach>;
}

template <typename T>
auto append_kernel(bool pairs, bool axes, int each) {
  return each == 1 ? append_kernel<T, 1>(pairs, axes) : append_kernel<T, 2>(pairs, axes);
}

}  // namespace
}  // namespace cpkv

extern "C" int cpkv_append_rotary(int64_t n_tokens, int page_size, int cp_size, int dtype, int q_heads, int kv_heads,
                                  int key_dim, int value_dim, int64_t row_bytes, int64_t key_offset,
                                  int64_t value_offset, void *const *h_pools, const int64_t *h_pool_cap_pages,
                                  const void *d_k, int64_t k_stride, const void *d_v, int64_t v_stride,
                                  const void *d_q, int64_t q_stride, void *d_q_out, int64_t q_out_stride,
                                  const int64_t *d_slots, const int32_t *d_positions, int64_t position_stride,
                                  int n_axes, const uint8_t *h_axis_of_freq, const float *d_cos_sin,
                                  int64_t max_position, int rot_dim, int flags, int32_t *d_status,
                                  cpkv_stream_t stream) {
  using namespace cpkv;
  AppendArgs args;
  args.n_tokens = n_tokens;
  args.dtype = dtype;
  args.q_heads = q_heads;
  args.kv_heads = kv_heads;
  args.key_dim = key_dim;
  args.value_dim = value_dim;
  args.d_k = d_k;
  args.d_v = d_v;
  args.d_q = d_q;
  args.d_q_out = d_q_out;
  args.k_stride = k_stride;
  args.v_stride = v_stride;
  args.q_stride = q_stride;
  args.q_out_stride = q_out_stride;
  args.d_slots = d_slots;
  args.d_positions = d_positions;
  args.position_stride = position_stride;
  args.n_axes = n_axes;
  args.h_axis_of_freq = h_axis_of_freq;
  args.d_cos_sin = d_cos_sin;
  args.max_position = max_position;
  args.rot_dim = rot_dim;
  args.d_status = d_status;
  if (flags & ~(CPKV_ROTARY_INTERLEAVED | CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_append_sizes(args);
  if (rc != CPKV_OK) return rc;
  AppendParams p = {};
  rc = paged_pools(&p.pools, page_size, cp_size, row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  const int64_t key_bytes = (int64_t)kv_heads * key_dim * 2, value_bytes = (int64_t)kv_heads * value_dim * 2;
  if (key_offset < 0 || value_offset < 0 || key_offset % 16 != 0 || value_offset % 16 != 0) return CPKV_ERR_ARG;
  if (key_offset + key_bytes > row_bytes || value_offset + value_bytes > row_bytes) return CPKV_ERR_ARG;
  if (key_offset < value_offset + value_bytes && value_offset < key_offset + key_bytes) return CPKV_ERR_ARG;
  rc = check_append_axes(args);
  if (rc != CPKV_OK || n_tokens == 0) return rc;
  rc = fill_append(&p, args);
  if (rc != CPKV_OK) return rc;
  p.k_off = key_offset;
  p.v_off = value_offset;
  p.value_chunks = kv_heads * value_dim / 8;
  const int head_units = (key_dim + 15) / 16;
  // Two heads a thread once that leaves every SM its 1024 threads, one before.
  // 44600 tokens of 32 + 8 heads of 128, all of a head rotated: 168 us with two (6.5
  // TB/s, 96% of the measured copy rate), 182 with one; four need registers that halve
  // the threads of an SM and lost to two.  512 tokens: 6.2 us with either.
  const int64_t units = n_tokens * ((int64_t)p.heads * head_units + p.value_chunks);
  const int each = units >= (int64_t)device_sm_count() * 2 * 1024 ? 2 : 1;
  p.head_groups = (int)ceil_div(p.heads, each);
  p.value_groups = (int)ceil_div(p.value_chunks, each);
  p.rotated = p.head_groups * head_units;
  p.head_units = fast_div((uint32_t)head_units);
  p.threads = fast_div((uint32_t)(p.rotated + p.value_groups));
  const bool pairs = flags & CPKV_ROTARY_INTERLEAVED, axes = n_axes > 1;
  auto kernel = dtype == CPKV_BF16 ? append_kernel<__nv_bfloat16>(pairs, axes, each) : append_kernel<__half>(pairs, axes, each);
  const int grid = persistent_grid((const void *)kernel, kAppendThreads, 0, 16, ceil_div(n_tokens * (int64_t)p.threads.d, kAppendThreads));
  return launch_kernel(kernel, dim3(grid), dim3(kAppendThreads), 0, false, (cudaStream_t)stream, p);
}
