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

constexpr int kThreads = 128;
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
  int n_tokens, q_heads, heads, key_dim, half, n_axes;  // heads: query and key heads
  int value_chunks;                                     // 16-byte chunks of a token's values
  int head_groups, value_groups;                        // a thread's heads (chunks) are this far apart
  int rotated;     // threads of a token that work on heads: head_groups * head_units
  FastDiv threads, head_units;  // threads of a token; units of a head
  alignas(4) uint8_t axis[kMaxHalf];
};

// One unit of work: unit u of token n, and what the token says of itself.
template <bool kAxes>
struct Work {
  int64_t id;
  int n, u;
  int64_t slot;
  int pos[kAxes ? kMaxAxes : 1];

  CPKV_DEV int64_t position(uint32_t axis) const {
    if constexpr (kAxes) return axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
    return pos[0];
  }
  // Whether every position of the token lies in the table: a token that fails is
  // dropped whole.
  CPKV_DEV bool positions_ok(const AppendParams &p) const {
    bool ok = pos[0] >= 0 && pos[0] < p.max_pos;
    if constexpr (kAxes) {
#pragma unroll
      for (int a = 1; a < kMaxAxes; ++a) ok &= pos[a] >= 0 && pos[a] < p.max_pos;
    }
    return ok;
  }
};

template <bool kAxes>
CPKV_DEV Work<kAxes> find_work(const AppendParams &p, int64_t id, int64_t total) {
  Work<kAxes> w;
  w.id = id;
  if (id >= total) return w;
  w.n = id < INT32_MAX ? div_by((int)id, p.threads) : (int)(id / p.threads.d);
  w.u = (int)(id - (int64_t)w.n * p.threads.d);
  w.slot = p.slots[w.n];
  w.pos[0] = p.positions[w.n];
  if constexpr (kAxes) {
#pragma unroll
    for (int a = 1; a < kMaxAxes; ++a) w.pos[a] = a < p.n_axes ? p.positions[a * p.pos_stride + w.n] : 0;
  }
  return w;
}

// Four cosines and sines, of frequencies f .. f + 3.
template <bool kAxes>
CPKV_DEV void angles4(const AppendParams &p, const Work<kAxes> &w, int f, float *c, float *s) {
  const int rot = 2 * p.half;
  uint32_t axes = 0;
  if (kAxes) axes = *reinterpret_cast<const uint32_t *>(p.axis + f);
  if (!kAxes || axes == (axes & 0xff) * 0x01010101u) {
    const float *const row = p.table + w.position(axes & 0xff) * rot + f;
    const float4 cs = __ldg(reinterpret_cast<const float4 *>(row));
    const float4 sn = __ldg(reinterpret_cast<const float4 *>(row + p.half));
    c[0] = cs.x, c[1] = cs.y, c[2] = cs.z, c[3] = cs.w;
    s[0] = sn.x, s[1] = sn.y, s[2] = sn.z, s[3] = sn.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float *const row = p.table + w.position(axes >> (8 * i) & 0xff) * rot + f + i;
    c[i] = __ldg(row);
    s[i] = __ldg(row + p.half);
  }
}

// Row of a slot in the pools; null (with a status bit) where its page is
// outside them, null for padding.
CPKV_DEV char *slot_row(const AppendParams &p, int64_t slot, bool reports) {
  if (slot < 0) return nullptr;
  const int64_t page = slot < INT32_MAX ? div_by((int)slot, p.pools.page_size) : slot / p.pools.page_size.d;
  char *base = page <= INT32_MAX ? page_address(p.pools, (int)page) : nullptr;
  if (base == nullptr) {
    if (reports) raise_status(p.status, CPKV_STATUS_PAGE_OOB);
    return nullptr;
  }
  return base + (slot - page * p.pools.page_size.d) * p.pools.row_bytes;
}

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
    if (!turns) {
      *reinterpret_cast<uint4 *>(dst + a0) = x0[e];
      if (two) *reinterpret_cast<uint4 *>(dst + a1) = x1[e];
      continue;
    }
    uint32_t y0[4] = {0, 0, 0, 0}, y1[4] = {0, 0, 0, 0};
    if (ok) {
      const uint32_t w0[4] = {x0[e].x, x0[e].y, x0[e].z, x0[e].w}, w1[4] = {x1[e].x, x1[e].y, x1[e].z, x1[e].w};
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
    }
    *reinterpret_cast<uint4 *>(dst + a0) = make_uint4(y0[0], y0[1], y0[2], y0[3]);
    *reinterpret_cast<uint4 *>(dst + a1) = make_uint4(y1[0], y1[1], y1[2], y1[3]);
  }
}

// A grid that stays resident walks the units; a unit's token is looked up one step
// ahead.  Blocks of their own for every 128 units spent a seventh of their time on
// coming and going.
template <typename T, bool kPairs, bool kAxes, int kEach>
__global__ void __launch_bounds__(kThreads) append_rotary_kernel(const __grid_constant__ AppendParams p) {
  const int64_t total = (int64_t)p.n_tokens * p.threads.d, step = (int64_t)gridDim.x * kThreads;
  Work<kAxes> w = find_work<kAxes>(p, (int64_t)blockIdx.x * kThreads + threadIdx.x, total);
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
  p.heads = q_heads + kv_heads;
  p.key_dim = key_dim;
  p.half = rot_dim / 2;
  p.n_axes = n_axes;
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
  const int grid = persistent_grid((const void *)kernel, kThreads, 0, 16, ceil_div(n_tokens * (int64_t)p.threads.d, kThreads));
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), 0, false, (cudaStream_t)stream, p);
}
