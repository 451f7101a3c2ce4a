// What the appends of new tokens share: their arguments and checks, units of
// work, the table's angles, rows by slot.
#pragma once

#include "paged.cuh"

namespace cpkv {

constexpr int kAppendThreads = 128;
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
  if constexpr (kAxes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float *const row = p.table + w.position(axes >> (8 * i) & 0xff) * rot + f + i;
      c[i] = __ldg(row);
      s[i] = __ldg(row + p.half);
    }
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

// Rotates the 16 elements of a unit by its 8 frequencies: one vector of first and one
// of second elements, or (kPairs) two of pairs, each word a pair.
template <typename T, bool kPairs>
CPKV_DEV void rotate_unit(uint4 &x0, uint4 &x1, const float *c, const float *s) {
  const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
  uint32_t y0[4], y1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack2<T>(w0[i]), b = unpack2<T>(w1[i]);
    if (kPairs) {  // a of frequency i, b of frequency i + 4
      y0[i] = pack2<T>(a.x * c[i] - a.y * s[i], a.y * c[i] + a.x * s[i]);
      y1[i] = pack2<T>(b.x * c[i + 4] - b.y * s[i + 4], b.y * c[i + 4] + b.x * s[i + 4]);
    } else {
      const int j = 2 * i;
      y0[i] = pack2<T>(a.x * c[j] - b.x * s[j], a.y * c[j + 1] - b.y * s[j + 1]);
      y1[i] = pack2<T>(b.x * c[j] + a.x * s[j], b.y * c[j + 1] + a.y * s[j + 1]);
    }
  }
  x0 = make_uint4(y0[0], y0[1], y0[2], y0[3]);
  x1 = make_uint4(y1[0], y1[1], y1[2], y1[3]);
}

// What an append's entry point is told, beside the pools and where a row keeps what.
struct AppendArgs {
  int64_t n_tokens;
  int dtype, q_heads, kv_heads, key_dim, value_dim;
  const void *d_k, *d_v, *d_q;
  void *d_q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  const int64_t *d_slots;
  const int32_t *d_positions;
  int64_t position_stride;
  int n_axes;
  const uint8_t *h_axis_of_freq;
  const float *d_cos_sin;
  int64_t max_position;
  int rot_dim;
  int32_t *d_status;
};

// Sizes, before the pools are looked at.
inline int check_append_sizes(const AppendArgs &a) {
  if (a.n_tokens < 0 || a.q_heads < 0 || a.kv_heads < 1 || a.key_dim <= 0 || a.value_dim <= 0 || a.rot_dim < 0) return CPKV_ERR_ARG;
  if (a.dtype != CPKV_BF16 && a.dtype != CPKV_FP16) return CPKV_ERR_ARG;
  if (a.key_dim % 8 != 0 || a.value_dim % 8 != 0 || a.rot_dim % 16 != 0 || a.rot_dim > a.key_dim) return CPKV_ERR_ARG;
  if (a.rot_dim > 2 * kMaxHalf || a.key_dim > 4096 || a.value_dim > 4096 || a.kv_heads > 1024 || a.q_heads > 1024)
    return CPKV_ERR_LIMIT;
  if (a.n_tokens > INT32_MAX || a.max_position > INT32_MAX) return CPKV_ERR_LIMIT;
  return CPKV_OK;
}

inline int check_append_axes(const AppendArgs &a) {
  if (a.n_axes < 1 || a.n_axes > kMaxAxes) return CPKV_ERR_ARG;
  if (a.n_axes > 1 && a.h_axis_of_freq == nullptr && a.rot_dim > 0) return CPKV_ERR_ARG;
  return CPKV_OK;
}

// Pointers and strides of at least one token, and what the kernels take of them.
inline int fill_append(AppendParams *p, const AppendArgs &a) {
  if (a.d_k == nullptr || a.d_v == nullptr || a.d_slots == nullptr || a.d_positions == nullptr || a.d_status == nullptr)
    return CPKV_ERR_ARG;
  if (a.rot_dim > 0 && (a.d_cos_sin == nullptr || a.max_position < 1)) return CPKV_ERR_ARG;
  if (a.q_heads > 0 && (a.d_q == nullptr || a.d_q_out == nullptr)) return CPKV_ERR_ARG;
  if (!aligned16(a.d_k) || !aligned16(a.d_v) || !aligned16(a.d_cos_sin)) return CPKV_ERR_ARG;
  if (a.k_stride < a.kv_heads * (int64_t)a.key_dim || a.v_stride < a.kv_heads * (int64_t)a.value_dim || a.k_stride % 8 != 0 ||
      a.v_stride % 8 != 0)
    return CPKV_ERR_ARG;
  if (a.q_heads > 0 && (!aligned16(a.d_q) || !aligned16(a.d_q_out) || a.q_stride % 8 != 0 || a.q_out_stride % 8 != 0 ||
                        a.q_stride < a.q_heads * (int64_t)a.key_dim || a.q_out_stride < a.q_heads * (int64_t)a.key_dim))
    return CPKV_ERR_ARG;
  if (a.n_axes > 1 && a.position_stride < a.n_tokens) return CPKV_ERR_ARG;
  for (int i = 0; i < a.rot_dim / 2 && a.n_axes > 1; ++i) {
    if (a.h_axis_of_freq[i] >= a.n_axes) return CPKV_ERR_ARG;
    p->axis[i] = a.h_axis_of_freq[i];
  }
  p->q = static_cast<const char *>(a.d_q);
  p->k = static_cast<const char *>(a.d_k);
  p->v = static_cast<const char *>(a.d_v);
  p->q_out = static_cast<char *>(a.d_q_out);
  p->slots = a.d_slots;
  p->positions = a.d_positions;
  p->table = a.d_cos_sin;
  p->status = a.d_status;
  p->q_stride = a.q_stride * 2;
  p->k_stride = a.k_stride * 2;
  p->v_stride = a.v_stride * 2;
  p->q_out_stride = a.q_out_stride * 2;
  p->pos_stride = a.position_stride;
  p->max_pos = a.rot_dim > 0 ? a.max_position : INT64_MAX;
  p->n_tokens = (int)a.n_tokens;
  p->q_heads = a.q_heads;
  p->heads = a.q_heads + a.kv_heads;
  p->key_dim = a.key_dim;
  p->half = a.rot_dim / 2;
  p->n_axes = a.n_axes;
  return CPKV_OK;
}

}  // namespace cpkv
