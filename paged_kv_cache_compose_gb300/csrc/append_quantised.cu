// cpkv_append_quantised: new keys and values into quantised rows, keys (and
// queries beside them) rotated by their positions on the way.
//
// A rotated key element is y = a c - b s (or b c + a s).  It is rounded to 16 bits
// nowhere on its way to e4m3, and not to 32 either in a way that shows: next to the
// border between two e4m3 numbers a product rounded to 32 bits can fall on the other
// side (one element in about 2^19), and the row would depend on the order of three
// instructions.  So products are held as pairs (a rounded product and its exact rest),
// and their sum is rounded "to odd": a 32-bit number whose last bit says that
// something follows rounds to e4m3 as the exact sum does.  Some twenty instructions
// more an element of the keys; bytes bound the call all the same (44600 tokens of 32 + 8
// heads of 128 in fp16, half of a head rotated).
#include "append.cuh"
#include "quantised.cuh"

namespace cpkv {
namespace {

struct QuantisedParams {
  AppendParams a;
  int64_t ks_off, vs_off;  // bytes of the scales in a row
  int value_first;         // first thread of a token that works on values
  int value_units;         // 16 elements each
  int key_heads_kept;      // keys stay in 16 bits
  int group_threads;       // threads of a group of values: 8, or 4
  int key_threads;         // of a key head
  FastDiv by_group;
};

// x y exactly, as a rounded product and the rest.
struct Exact {
  float hi, lo;
};
CPKV_DEV Exact product(float x, float y) {
  const float p = __fmul_rn(x, y);
  return Exact{p, __fmaf_rn(x, y, -p)};
}
CPKV_DEV Exact sum(float x, float y) {
  const float s = __fadd_rn(x, y), z = __fsub_rn(s, x);
  return Exact{s, __fadd_rn(__fsub_rn(x, __fsub_rn(s, z)), __fsub_rn(y, z))};
}

// p + q rounded to odd: towards zero, the last bit set unless the sum is exact.
CPKV_DEV float sum_to_odd(Exact p, Exact q) {
  const Exact top = sum(p.hi, q.hi);
  const Exact r = sum(top.hi, __fadd_rn(top.lo, __fadd_rn(p.lo, q.lo)));
  uint32_t bits = __float_as_uint(r.hi);
  if (r.lo != 0.f) bits = (bits - ((__float_as_uint(r.lo) ^ bits) >> 31)) | 1u;
  return __uint_as_float(bits);
}

// The largest of a group's threads, which lie side by side.
CPKV_DEV float largest_of(float x, int threads) {
  const uint32_t first = (threadIdx.x & 31) & ~(uint32_t)(threads - 1), mask = ((1u << threads) - 1) << first;
  x = fmaxf(x, __shfl_xor_sync(mask, x, 1));
  x = fmaxf(x, __shfl_xor_sync(mask, x, 2));
  if (threads == 8) x = fmaxf(x, __shfl_xor_sync(mask, x, 4));
  return x;
}

// The largest magnitude of 16 finite elements; infinite ones become NaNs.
CPKV_DEV float largest_of16(float (&y)[16]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = finite_or_nan(y[i]);
    top = fmaxf(top, fabsf(y[i]));  // a NaN is no largest
  }
  return top;
}

CPKV_DEV uint2 pack8(const float *y, float f) {
  return make_uint2(pack_e4m3(y[0] * f, y[1] * f, y[2] * f, y[3] * f), pack_e4m3(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
}

template <typename T>
CPKV_DEV void unpack8(const uint4 &v, float *y) {
  const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y), c = unpack2<T>(v.z), d = unpack2<T>(v.w);
  y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y, y[4] = c.x, y[5] = c.y, y[6] = d.x, y[7] = d.y;
}

// A thread's unit is 16 elements: of a head, 8 frequencies' elements (two 16-byte
// vectors) or 16 plain ones; of the values, 16 in a row.  A group's threads lie side by
// side in a warp, a token's threads come in eights, so that the largest magnitude is
// found by shuffles and each row is written once.
template <typename T, bool kPairs, bool kAxes, int kEach>
CPKV_DEV void quantise_work(const QuantisedParams &p, const Work<kAxes> &w) {
  const AppendParams &a = p.a;
  const int n = w.n, u = w.u;
  const bool ok = w.positions_ok(a);
  if (u >= a.rotated) {  // values
    const int first = u - p.value_first;
    if (first < 0) return;  // between the heads and the values
    const char *src = a.v + n * a.v_stride;
    uint4 x[kEach][2];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int c = first + e * a.value_groups;
      if (c < p.value_units) x[e][0] = ld_stream16(src + c * 32), x[e][1] = ld_stream16(src + c * 32 + 16);
    }
    char *const row = ok ? slot_row(a, w.slot, false) : nullptr;
    if (row == nullptr) return;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int c = first + e * a.value_groups;
      if (c >= p.value_units) continue;
      float y[16];
      unpack8<T>(x[e][0], y);
      unpack8<T>(x[e][1], y + 8);
      const GroupScale g = group_scale(largest_of(largest_of16(y), p.group_threads));
      const uint2 lo = pack8(y, g.inverse), hi = pack8(y + 8, g.inverse);
      *reinterpret_cast<uint4 *>(row + a.v_off + c * 16) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      if ((c & (p.group_threads - 1)) == 0)
        *reinterpret_cast<float *>(row + p.vs_off + div_by(c, p.by_group) * 4) = g.scale;
    }
    return;
  }

  const int first = div_by(u, a.head_units), unit = u - first * (int)a.head_units.d;
  const bool turns = unit * 8 < a.half;
  const int head_bytes = a.key_dim * 2;
  const int a0 = turns && !kPairs ? unit * 16 : unit * 32;  // plain units follow the rotated 2 half elements
  const int a1 = turns && !kPairs ? a0 + a.half * 2 : a0 + 16;
  const bool two = a1 < head_bytes;
  const char *const q = a.q + n * a.q_stride, *const k = a.k + n * a.k_stride;
  char *const q_out = a.q_out + n * a.q_out_stride;
  uint4 x0[kEach], x1[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int head = first + e * a.head_groups;
    if (head >= a.heads) continue;
    const char *src = head < a.q_heads ? q + head * head_bytes : k + (head - a.q_heads) * head_bytes;
    x0[e] = ld_stream16(src + a0);
    if (two) x1[e] = ld_stream16(src + a1);
  }
  float c[8], s[8];
  if (turns && ok) {
    angles4<kAxes>(a, w, unit * 8, c, s);
    angles4<kAxes>(a, w, unit * 8 + 4, c + 4, s + 4);
  }
  if (!ok && u == 0) raise_status(a.status, CPKV_STATUS_POS_OOB);
  char *const row = ok ? slot_row(a, w.slot, u == 0) : nullptr;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int head = first + e * a.head_groups;
    if (head >= a.heads) continue;
    if (head >= a.q_heads && !p.key_heads_kept) {  // a quantised key head
      if (row == nullptr) continue;
      float v[16], y[16];  // a thread's first, then its second vector
      unpack8<T>(x0[e], v);
      unpack8<T>(x1[e], v + 8);
      if (turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int one = kPairs ? 2 * i : i, two_ = kPairs ? 2 * i + 1 : i + 8;
          const Exact ac = product(v[one], c[i]), bc = product(v[two_], c[i]);
          const Exact as = product(v[one], s[i]), bs = product(v[two_], s[i]);
          y[one] = sum_to_odd(ac, Exact{-bs.hi, -bs.lo});
          y[two_] = sum_to_odd(bc, as);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = v[i];
      }
      const GroupScale g = group_scale(largest_of(largest_of16(y), p.key_threads));
      char *const dst = row + a.k_off + (head - a.q_heads) * a.key_dim;
      *reinterpret_cast<uint2 *>(dst + (a0 >> 1)) = pack8(y, g.inverse);
      *reinterpret_cast<uint2 *>(dst + (a1 >> 1)) = pack8(y + 8, g.inverse);
      if (unit == 0) *reinterpret_cast<float *>(row + p.ks_off + (head - a.q_heads) * 4) = g.scale;
      continue;
    }
    char *dst;
    if (head < a.q_heads) {
      dst = q_out + head * head_bytes;
      if (!ok) x0[e] = x1[e] = make_uint4(0, 0, 0, 0);
    } else {
      if (row == nullptr) continue;
      dst = row + a.k_off + (head - a.q_heads) * head_bytes;
    }
    if (turns && ok) rotate_unit<T, kPairs>(x0[e], x1[e], c, s);
    *reinterpret_cast<uint4 *>(dst + a0) = x0[e];
    if (two) *reinterpret_cast<uint4 *>(dst + a1) = x1[e];
  }
}

template <typename T, bool kPairs, bool kAxes, int kEach>
__global__ void __launch_bounds__(kAppendThreads) append_quantised_kernel(const __grid_constant__ QuantisedParams p) {
  const int64_t total = (int64_t)p.a.n_tokens * p.a.threads.d, step = (int64_t)gridDim.x * kAppendThreads;
  Work<kAxes> w = find_work<kAxes>(p.a, (int64_t)blockIdx.x * kAppendThreads + threadIdx.x, total);
  while (w.id < total) {  // a token's threads come in eights: a group's go on together
    const Work<kAxes> next = find_work<kAxes>(p.a, w.id + step, total);
    quantise_work<T, kPairs, kAxes, kEach>(p, w);
    w = next;
  }
}

template <typename T, int kEach>
auto quantised_kernel(bool pairs, bool axes) {
  if (pairs) return axes ? append_quantised_kernel<T, true, true, kEach> : append_quantised_kernel<T, true, false, kEach>;
  return axes ? append_quantised_kernel<T, false, true, kEach> : append_quantised_kernel<T, false, false, kEach>;
}

template <typename T>
auto quantised_kernel(bool pairs, bool axes, int each) {
  return each == 1 ? quantised_kernel<T, 1>(pairs, axes) : quantised_kernel<T, 2>(pairs, axes);
}

}  // namespace
}  // namespace cpkv

extern "C" int cpkv_append_quantised(int64_t n_tokens, int page_size, int cp_size, int dtype, int q_heads,
                                     const cpkv_quantised_row *h_row, void *const *h_pools,
                                     const int64_t *h_pool_cap_pages, const void *d_k, int64_t k_stride,
                                     const void *d_v, int64_t v_stride, const void *d_q, int64_t q_stride,
                                     void *d_q_out, int64_t q_out_stride, const int64_t *d_slots,
                                     const int32_t *d_positions, int64_t position_stride, int n_axes,
                                     const uint8_t *h_axis_of_freq, const float *d_cos_sin, int64_t max_position,
                                     int rot_dim, int flags, int32_t *d_status, cpkv_stream_t stream) {
  using namespace cpkv;
  if (flags & ~(CPKV_ROTARY_INTERLEAVED | CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_quantised_row(h_row);
  if (rc != CPKV_OK) return rc;
  const cpkv_quantised_row &row = *h_row;
  AppendArgs args;
  args.n_tokens = n_tokens;
  args.dtype = dtype;
  args.q_heads = q_heads;
  args.kv_heads = row.kv_heads;
  args.key_dim = row.key_dim;
  args.value_dim = row.value_dim;
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
  rc = check_append_sizes(args);
  if (rc != CPKV_OK) return rc;
  QuantisedParams p = {};
  rc = paged_pools(&p.a.pools, page_size, cp_size, row.row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  rc = check_append_axes(args);
  if (rc != CPKV_OK || n_tokens == 0) return rc;
  rc = fill_append(&p.a, args);
  if (rc != CPKV_OK) return rc;
  p.a.k_off = row.key_offset;
  p.a.v_off = row.value_offset;
  p.ks_off = row.key_scale_offset;
  p.vs_off = row.value_scale_offset;
  p.key_heads_kept = row.keep_keys != 0;
  p.group_threads = value_group(row) / 16;
  p.by_group = fast_div((uint32_t)p.group_threads);
  p.key_threads = row.key_dim / 16;
  p.value_units = row.kv_heads * row.value_dim / 16;
  const int head_units = (row.key_dim + 15) / 16;
  // Two heads (16 values twice) a thread once that leaves every SM its 1024 threads,
  // one before, as in the append without quantisation.
  const int64_t units = n_tokens * ((int64_t)p.a.heads * head_units + p.value_units);
  const int each = units >= (int64_t)device_sm_count() * 2 * 1024 ? 2 : 1;
  p.a.head_groups = (int)ceil_div(p.a.heads, each);
  p.a.value_groups = (int)ceil_div(ceil_div(p.value_units, each), 8) * 8;
  p.a.rotated = p.a.head_groups * head_units;
  p.value_first = (int)ceil_div(p.a.rotated, 8) * 8;
  p.a.head_units = fast_div((uint32_t)head_units);
  p.a.threads = fast_div((uint32_t)(p.value_first + p.a.value_groups));
  const bool pairs = flags & CPKV_ROTARY_INTERLEAVED, axes = n_axes > 1;
  auto kernel = dtype == CPKV_BF16 ? quantised_kernel<__nv_bfloat16>(pairs, axes, each) : quantised_kernel<__half>(pairs, axes, each);
  const int grid = persistent_grid((const void *)kernel, kAppendThreads, 0, 16, ceil_div(n_tokens * (int64_t)p.a.threads.d, kAppendThreads));
  return launch_kernel(kernel, dim3(grid), dim3(kAppendThreads), 0, false, (cudaStream_t)stream, p);
}
