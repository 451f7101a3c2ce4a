// cpkv_append_rotary: new keys and values into the paged pools, keys (and
// queries beside them) rotated by their positions on the way.
//
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a
//
// for each pair (x1, x2) of frequency i, with cos a and sin a of row
// pos[axis(i)] of the caller's table.  Three multiplications and additions per
// element, so bytes bound it (and, for a few tokens, the launch): every row is
// read once and written once, products are held in 32 bits and rounded once.
#include "paged.cuh"

namespace cpkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;
constexpr int kMaxHalf = 128;  // frequencies: rot_dim / 2

struct AppendParams {
  PagedPools pools;
  const char *q, *k, *v;
  char *q_out;
  const int64_t *slots;
  const int32_t *positions;
  const float *table;
  int32_t *status;
  int64_t q_stride, k_stride, v_stride, q_out_stride, pos_stride;  // bytes between tokens (positions: elements)
  int64_t max_pos, k_off, v_off;
  int n_tokens, q_heads, kv_heads, key_dim, half, n_axes;
  int units;       // work units of a token
  int key_units;   // of them in rotated heads: (q_heads + kv_heads) * head_units
  FastDiv units_div, head_units;
  uint8_t axis[kMaxHalf];
};

// Cosines and sines of frequencies f0 .. f0 + 7.
template <bool kAxes>
CPKV_DEV bool angles(const AppendParams &p, int n, int f0, float c[8], float s[8]) {
  const int rot = 2 * p.half;
  bool same = true;
  if (kAxes) {
#pragma unroll
    for (int i = 1; i < 8; ++i) same &= p.axis[f0 + i] == p.axis[f0];
  }
  if (!kAxes || same) {
    const int a = kAxes ? p.axis[f0] : 0;
    const int64_t pos = p.positions[a * p.pos_stride + n];
    if (pos < 0 || pos >= p.max_pos) return false;
    const float4 *row = reinterpret_cast<const float4 *>(p.table + pos * rot + f0);
    const float4 *sin_row = reinterpret_cast<const float4 *>(p.table + pos * rot + p.half + f0);
    const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(sin_row), s1 = __ldg(sin_row + 1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
    return true;
  }
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t pos = p.positions[p.axis[f0 + i] * p.pos_stride + n];
    const bool in = pos >= 0 && pos < p.max_pos;
    ok &= in;
    c[i] = in ? __ldg(p.table + pos * rot + f0 + i) : 0.f;
    s[i] = in ? __ldg(p.table + pos * rot + p.half + f0 + i) : 0.f;
  }
  return ok;
}

// Whether every position of token n lies in the table: a token that fails is
// dropped whole, so each of its units decides alike.
CPKV_DEV bool positions_ok(const AppendParams &p, int n) {
  bool ok = true;
  for (int a = 0; a < p.n_axes; ++a) {
    const int64_t pos = p.positions[a * p.pos_stride + n];
    ok &= pos >= 0 && pos < p.max_pos;
  }
  return ok;
}

// One unit per thread.  Units of a token, in order: per query head then per
// key head, half / 8 units of 16 rotated elements (8 frequencies; two 16-byte
// vectors) and (key_dim - 2 half) / 8 units of 8 plain ones; then the values,
// 8 elements each.  A token's units sit side by side, so warps read and write
// whole heads; the table rows that its heads share come from L1.
template <typename T, bool kPairs, bool kAxes>
__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const __grid_constant__ AppendParams p) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int n, u;
  if (id < INT32_MAX) {
    n = div_by((int)id, p.units_div);
    u = (int)id - n * p.units;
  } else {
    n = (int)(id / p.units);
    u = (int)(id - (int64_t)n * p.units);
  }
  if (n >= p.n_tokens) return;
  int head = 0, in_head = 0;
  if (u < p.key_units) {
    head = div_by(u, p.head_units);
    in_head = u - head * (int)p.head_units.d;
  }
  const bool is_q = u < p.key_units && head < p.q_heads;
  const bool ok = positions_ok(p, n);
  char *dst;
  if (is_q) {
    dst = p.q_out + n * p.q_out_stride + (int64_t)head * p.key_dim * 2;
  } else {
    const int64_t slot = p.slots[n];
    if (slot < 0 || !ok) {
      if (slot >= 0 && u == p.key_units) raise_status(p.status, CPKV_STATUS_POS_OOB);
      return;
    }
    const int64_t page = slot < INT32_MAX ? div_by((int)slot, p.pools.page_size) : slot / p.pools.page_size.d;
    char *base = page <= INT32_MAX ? page_address(p.pools, (int)page) : nullptr;
    if (base == nullptr) {
      if (u == p.key_units) raise_status(p.status, CPKV_STATUS_PAGE_OOB);
      return;
    }
    dst = base + (slot - page * p.pools.page_size.d) * p.pools.row_bytes;
    if (u >= p.key_units) {  // a value vector
      const int64_t at = (int64_t)(u - p.key_units) * 16;
      *reinterpret_cast<uint4 *>(dst + p.v_off + at) = ld_stream16(p.v + n * p.v_stride + at);
      return;
    }
    dst += p.k_off + (int64_t)(head - p.q_heads) * p.key_dim * 2;
  }
  const char *src = is_q ? p.q + n * p.q_stride + (int64_t)head * p.key_dim * 2
                         : p.k + n * p.k_stride + (int64_t)(head - p.q_heads) * p.key_dim * 2;
  if (!ok) {  // a query of a dropped token
    if (u == 0) raise_status(p.status, CPKV_STATUS_POS_OOB);
    if (in_head * 8 >= p.half) {
      *reinterpret_cast<uint4 *>(dst + (2 * p.half + (in_head - p.half / 8) * 8) * 2) = make_uint4(0, 0, 0, 0);
    } else {
      *reinterpret_cast<uint4 *>(dst + in_head * 32) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4 *>(dst + in_head * 32 + 16) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  if (in_head * 8 >= p.half) {  // elements past the rotated ones
    const int at = (2 * p.half + (in_head - p.half / 8) * 8) * 2;
    *reinterpret_cast<uint4 *>(dst + at) = ld_stream16(src + at);
    return;
  }
  const int f0 = in_head * 8;
  const int a0 = kPairs ? f0 * 4 : f0 * 2, a1 = kPairs ? a0 + 16 : a0 + p.half * 2;
  const uint4 x0 = ld_stream16(src + a0), x1 = ld_stream16(src + a1);
  float c[8], s[8];
  if (!angles<kAxes>(p, n, f0, c, s)) return;
  const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
  uint32_t y0[4], y1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack2<T>(w0[i]), b = unpack2<T>(w1[i]);
    if (kPairs) {  // each word is one pair: a of frequency i, b of frequency i + 4
      y0[i] = pack2<T>(a.x * c[i] - a.y * s[i], a.y * c[i] + a.x * s[i]);
      y1[i] = pack2<T>(b.x * c[i + 4] - b.y * s[i + 4], b.y * c[i + 4] + b.x * s[i + 4]);
    } else {
      const int j = 2 * i;
      y0[i] = pack2<T>(a.x * c[j] - b.x * s[j], a.y * c[j + 1] - b.y * s[j + 1]);
      y1[i] = pack2<T>(b.x * c[j] + a.x * s[j], b.y * c[j + 1] + a.y * s[j + 1]);
    }
  }
  *reinterpret_cast<uint4 *>(dst + a0) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
  *reinterpret_cast<uint4 *>(dst + a1) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
}

template <typename T>
auto append_kernel(bool pairs, bool axes) {
  if (pairs) return axes ? append_rotary_kernel<T, true, true> : append_rotary_kernel<T, true, false>;
  return axes ? append_rotary_kernel<T, false, true> : append_rotary_kernel<T, false, false>;
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
  if (n_tokens < 0 || q_heads < 0 || kv_heads < 1 || key_dim <= 0 || value_dim <= 0 || rot_dim < 0) return CPKV_ERR_ARG;
  if (dtype != CPKV_BF16 && dtype != CPKV_FP16) return CPKV_ERR_ARG;
  if (flags & ~(CPKV_ROTARY_INTERLEAVED | CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  if (key_dim % 8 != 0 || value_dim % 8 != 0 || rot_dim % 16 != 0 || rot_dim > key_dim) return CPKV_ERR_ARG;
  if (rot_dim > 2 * kMaxHalf || key_dim > 4096 || value_dim > 4096 || kv_heads > 1024 || q_heads > 1024)
    return CPKV_ERR_LIMIT;
  if (n_tokens > INT32_MAX || max_position > INT32_MAX) return CPKV_ERR_LIMIT;
  AppendParams p = {};
  const int rc = paged_pools(&p.pools, page_size, cp_size, row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  const int64_t key_bytes = (int64_t)kv_heads * key_dim * 2, value_bytes = (int64_t)kv_heads * value_dim * 2;
  if (key_offset < 0 || value_offset < 0 || key_offset % 16 != 0 || value_offset % 16 != 0) return CPKV_ERR_ARG;
  if (key_offset + key_bytes > row_bytes || value_offset + value_bytes > row_bytes) return CPKV_ERR_ARG;
  if (key_offset < value_offset + value_bytes && value_offset < key_offset + key_bytes) return CPKV_ERR_ARG;
  if (n_axes < 1 || n_axes > kMaxAxes) return CPKV_ERR_ARG;
  if (n_axes > 1 && h_axis_of_freq == nullptr && rot_dim > 0) return CPKV_ERR_ARG;
  if (n_tokens == 0) return CPKV_OK;
  if (d_k == nullptr || d_v == nullptr || d_slots == nullptr || d_positions == nullptr || d_status == nullptr)
    return CPKV_ERR_ARG;
  if (rot_dim > 0 && (d_cos_sin == nullptr || max_position < 1)) return CPKV_ERR_ARG;
  if (q_heads > 0 && (d_q == nullptr || d_q_out == nullptr)) return CPKV_ERR_ARG;
  if (!aligned16(d_k) || !aligned16(d_v) || !aligned16(d_cos_sin)) return CPKV_ERR_ARG;
  if (k_stride < kv_heads * (int64_t)key_dim || v_stride < kv_heads * (int64_t)value_dim || k_stride % 8 != 0 ||
      v_stride % 8 != 0)
    return CPKV_ERR_ARG;
  if (q_heads > 0 && (!aligned16(d_q) || !aligned16(d_q_out) || q_stride % 8 != 0 || q_out_stride % 8 != 0 ||
                      q_stride < q_heads * (int64_t)key_dim || q_out_stride < q_heads * (int64_t)key_dim))
    return CPKV_ERR_ARG;
  if (n_axes > 1 && position_stride < n_tokens) return CPKV_ERR_ARG;
  for (int i = 0; i < rot_dim / 2 && n_axes > 1; ++i) {
    if (h_axis_of_freq[i] >= n_axes) return CPKV_ERR_ARG;
    p.axis[i] = h_axis_of_freq[i];
  }
  p.q = static_cast<const char *>(d_q);
  p.k = static_cast<const char *>(d_k);
  p.v = static_cast<const char *>(d_v);
  p.q_out = static_cast<char *>(d_q_out);
  p.slots = d_slots;
  p.positions = d_positions;
  p.table = d_cos_sin;
  p.status = d_status;
  p.q_stride = q_stride * 2;
  p.k_stride = k_stride * 2;
  p.v_stride = v_stride * 2;
  p.q_out_stride = q_out_stride * 2;
  p.pos_stride = position_stride;
  p.max_pos = rot_dim > 0 ? max_position : INT64_MAX;
  p.k_off = key_offset;
  p.v_off = value_offset;
  p.n_tokens = (int)n_tokens;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.key_dim = key_dim;
  p.half = rot_dim / 2;
  p.n_axes = n_axes;
  p.head_units = fast_div((uint32_t)(rot_dim / 16 + (key_dim - rot_dim) / 8));
  p.key_units = (q_heads + kv_heads) * (int)p.head_units.d;
  p.units = p.key_units + kv_heads * value_dim / 8;
  p.units_div = fast_div((uint32_t)p.units);
  const int64_t blocks = ceil_div(n_tokens * p.units, kThreads);
  if (blocks > INT32_MAX) return CPKV_ERR_LIMIT;
  const bool pairs = flags & CPKV_ROTARY_INTERLEAVED, axes = n_axes > 1;
  return launch_kernel(dtype == CPKV_BF16 ? append_kernel<__nv_bfloat16>(pairs, axes) : append_kernel<__half>(pairs, axes),
                       dim3((unsigned)blocks), dim3(kThreads), 0, false, (cudaStream_t)stream, p);
}
