// cpkv_append_quantised: new keys and values into quantised rows, keys (and
// queries beside them) rotated by their positions on the way.
//
// A rotated key element is y = a c - b s (or b c + a s), and what is kept is e4m3 of y over the
// group's scale.  In 32 bits y is off by less than 2^-23 of |a c| + |b s|, which falls on the
// wrong side of a border between two e4m3 numbers for one element in about 2^18: the row
// would depend on the order of three instructions.  So each element is rounded from below and
// from above its error, and where the two differ it is worked out again in 64 bits (a whole head
// where its scale may differ, or 32 bits' range does not hold it): exact products, their sum rounded
// "to odd", towards zero with a last bit that says that something follows, which then rounds
// to e4m3 as the exact sum does.  Bytes bound the call (5.6 TB/s
// on 44600 tokens of 32 + 8 heads of 128, in 183 us) nearly as much as instructions do.
#include "append.cuh"
#include "quantised.cuh"

namespace cpkv {
namespace {

struct QuantisedParams {
  AppendParams a;
  int64_t ks_off, vs_off;  // bytes of the scales in a row
  int keys_kept;           // keys stay in 16 bits
  int lane_shift;          // 2^lane_shift lanes take a head, 16 elements each
  int group_threads;       // of a group of values: 8, or 4
  int value_units;         // 16 elements each
  // A token's work in turns of a warp: query heads, key heads, values; turn i is that of
  // warp i % parts of the token.
  int q_turns, k_turns, v_turns, k_first, v_first;  // k_first: q_turns % parts; v_first: (q_turns + k_turns) % parts
  FastDiv parts;
};

// a c + b s "rounded to odd": to 64 bits towards zero, the last bit set unless the sum is exact.
// The products are exact (11 and 24 bits of fraction at most, and far from the ends of the
// range), and so is the rest of their sum.
CPKV_DEV double turned_to_odd(float a, float c, float b, float s) {
  const double p = (double)a * c, q = (double)b * s, sum = __dadd_rn(p, q), z = __dsub_rn(sum, p);
  const double rest = __dadd_rn(__dsub_rn(p, __dsub_rn(sum, z)), __dsub_rn(q, z));
  long long bits = __double_as_longlong(sum);
  if (rest != 0 && fabs(sum) < INFINITY) bits = (bits - ((__double_as_longlong(rest) ^ bits) < 0 ? 1 : 0)) | 1;
  return __longlong_as_double(bits);
}

// The same number in 32 bits, rounded to odd.
CPKV_DEV float to_odd(double x) {
  const float y = __double2float_rz(x);
  return y == x ? y : __uint_as_float(__float_as_uint(y) | 1u);
}

// The largest of a group's threads, which lie side by side.
template <typename F>
CPKV_DEV F largest_of(F x, int threads) {
  const uint32_t first = (threadIdx.x & 31) & ~(uint32_t)(threads - 1), mask = ((1u << threads) - 1) << first;
  x = max(x, __shfl_xor_sync(mask, x, 1));
  x = max(x, __shfl_xor_sync(mask, x, 2));
  if (threads == 8) x = max(x, __shfl_xor_sync(mask, x, 4));
  return x;
}

// The largest magnitude of a group's finite elements, 16 of them this thread's.  Infinities
// and NaNs (acc + 0 y is one then) are rare: infinite ones become NaNs, and are no largest.
CPKV_DEV float largest_of16(float (&y)[16], int threads) {
  float top = fabsf(y[0]), marks = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = fmaxf(top, fabsf(y[i]));
    marks = __fmaf_rn(y[i], 0.f, marks);
  }
  if (marks != 0.f) {
    top = 0.f;
    for (int i = 0; i < 16; ++i) {
      y[i] = finite_or_nan(y[i]);
      top = fmaxf(top, fabsf(y[i]));
    }
  }
  return largest_of(top, threads);
}

// The same of 16-bit elements as they are, two at a time: their bits order like their
// magnitudes, infinities and NaNs last.
template <typename T>
CPKV_DEV bool largest_of16(const uint4 &a, const uint4 &b, int threads, float *top) {
  constexpr uint32_t kInfinite = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u, kAll = 0x7fff7fffu;
  const uint32_t w = __vmaxu2(__vmaxu2(__vmaxu2(a.x & kAll, a.y & kAll), __vmaxu2(a.z & kAll, a.w & kAll)),
                              __vmaxu2(__vmaxu2(b.x & kAll, b.y & kAll), __vmaxu2(b.z & kAll, b.w & kAll)));
  const uint32_t most = max(w & 0xffffu, w >> 16);
  *top = largest_of(unpack2<T>(most).x, threads);  // of NaNs none
  const uint32_t first = (threadIdx.x & 31) & ~(uint32_t)(threads - 1), mask = ((1u << threads) - 1) << first;
  return __any_sync(mask, most >= kInfinite) == 0;
}

CPKV_DEV uint2 pack8(const float *y, float f) {
  return make_uint2(pack_e4m3(y[0] * f, y[1] * f, y[2] * f, y[3] * f), pack_e4m3(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
}

// Whether a condition holds for all threads of a group.
CPKV_DEV bool all_of(bool ok, int threads) {
  const uint32_t first = (threadIdx.x & 31) & ~(uint32_t)(threads - 1), mask = ((1u << threads) - 1) << first;
  return __all_sync(mask, ok) != 0;
}

// Quantises a thread's 16 elements, each known to the error d of its pair: bytes of the least and of the
// most that it may be, and the group's scale.  False where that may depend on the errors too, an element is
// infinite or a NaN, or the errors are not relative ones because products leave the normal numbers: in a group that
// reaches 2^-100 an element of 2^-120 or more has an error of less than d also with what is lost below 2^-149, and a
// smaller one is e4m3's zero; of other groups only zeros are known.
template <bool kPairs>
CPKV_DEV bool quantise_between(const float *y, const float *d, int threads, GroupScale *g, uint32_t (&below)[4], uint32_t (&above)[4]) {
  float top = 0.f, off = 0.f, marks = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = fmaxf(top, fabsf(y[i]));
    marks = __fmaf_rn(y[i], 0.f, marks);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) off = fmaxf(off, d[i]);
  const float most = largest_of(top + off, threads), least = largest_of(top - off, threads);
  *g = group_scale(most);
  const float f = g->inverse;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    float a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 4 * w + k;
      const float z = y[i] * f, e = d[kPairs ? i / 2 : i % 8] * f;
      a[k] = z - e;
      b[k] = z + e;
    }
    below[w] = pack_e4m3(a[0], a[1], a[2], a[3]);
    above[w] = pack_e4m3(b[0], b[1], b[2], b[3]);
  }
  return marks == 0.f && (most >= 0x1p-100f || most == 0.f) && group_scale(least).scale == g->scale;
}

template <typename T>
CPKV_DEV void unpack8(const uint4 &v, float *y) {
  const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y), c = unpack2<T>(v.z), d = unpack2<T>(v.w);
  y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y, y[4] = c.x, y[5] = c.y, y[6] = d.x, y[7] = d.y;
}

struct ExactUnit {
  uint32_t bytes[4];
  float scale;
};

// A unit of a key head, the elements that are not known yet (a bit each) exactly, and the group's scale
// where that is not (`whole`, of all its threads).  Read again, apart and an element at a time, so that
// the usual way needs no registers for it.  64-bit operations are slow: with all of a head's elements so, the
// traced append took 259 us.
template <typename T, bool kPairs, bool kAxes>
__device__ __noinline__ ExactUnit exact_unit(const QuantisedParams &p, const Work<kAxes> &w, int head, int unit, bool whole, uint32_t unknown,
                                             ExactUnit known) {
  const AppendParams &a = p.a;
  const bool turns = unit * 8 < a.half;
  const int a0 = turns && !kPairs ? unit * 16 : unit * 32, a1 = turns && !kPairs ? a0 + a.half * 2 : a0 + 16;
  const char *const src = a.k + w.n * a.k_stride + head * (a.key_dim * 2);
  float v[16], c[8], s[8];
  unpack8<T>(ld_stream16(src + a0), v);
  unpack8<T>(ld_stream16(src + a1), v + 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;  // of elements that are not turned
  if (turns) {
    angles4<kAxes>(a, w, unit * 8, c, s);
    angles4<kAxes>(a, w, unit * 8 + 4, c + 4, s + 4);
  }
  struct Turn {
    float a, c, b, s;
  };
  auto turn_of = [&](int i) {  // element i is a c + b s
    const int k = kPairs ? i / 2 : i % 8, first = kPairs ? 2 * k : k, other = i == first ? first + (kPairs ? 1 : 8) : first;
    return Turn{v[i], c[k], turns ? v[other] : 0.f, i == first ? -s[k] : s[k]};
  };
  int e = (int)(__float_as_uint(known.scale) >> 23) - 127;
  if (whole) {
    double top = 0;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const Turn t = turn_of(i);
      const double y = fabs(turned_to_odd(t.a, t.c, t.b, t.s));
      if (y <= kMostQuantised) top = max(top, y);
    }
    e = group_exponent(largest_of(top, 1 << p.lane_shift));
    known.scale = __uint_as_float((uint32_t)(127 + e) << 23);
    unknown = 0xffffu;
  }
  const double inverse = __hiloint2double((1023 - e) << 20, 0);
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    if (!(unknown >> i & 1)) continue;
    const Turn t = turn_of(i);
    const double y = turned_to_odd(t.a, t.c, t.b, t.s);
    const float z = fabs(y) <= kMostQuantised ? to_odd(y * inverse) : NAN;
    const uint32_t byte = pack_e4m3(z, 0.f, 0.f, 0.f) & 0xffu;
    const int at = i % 4 * 8;
    known.bytes[i / 4] = (known.bytes[i / 4] & ~(0xffu << at)) | byte << at;
  }
  return known;
}

// A bit for each byte in which two words differ.
CPKV_DEV uint32_t differing(uint32_t x, uint32_t y) {
  const uint32_t d = x ^ y;
  return ((d & 0xffu) != 0) | ((d & 0xff00u) != 0) << 1 | ((d & 0xff0000u) != 0) << 2 | ((d & 0xff000000u) != 0) << 3;
}

// A warp takes a token, or one of `parts` shares of it where tokens are few: its row and
// angles are looked up once for all its heads.  A unit is 16 elements: of a head, 8
// frequencies' elements (two 16-byte vectors) or 16 plain ones; of the values, 16 in a
// row.  A group's threads lie side by side in a warp, so that its largest magnitude is found
// by shuffles and each row is written once.
template <typename T, bool kPairs, bool kAxes, int kAtOnce>
CPKV_DEV void quantise_token(const QuantisedParams &p, const Work<kAxes> &w, int part) {
  const AppendParams &a = p.a;
  const int n = w.n, lane = threadIdx.x & 31, parts = p.parts.d;
  const bool ok = w.positions_ok(a), reports = part == 0 && lane == 0;
  if (!ok && reports) raise_status(a.status, CPKV_STATUS_POS_OOB);
  char *const row = ok ? slot_row(a, w.slot, reports) : nullptr;
  const int unit = lane & ((1 << p.lane_shift) - 1), sub = lane >> p.lane_shift, heads = 32 >> p.lane_shift;  // of a turn
  const int head_bytes = a.key_dim * 2;
  const bool turns = unit * 8 < a.half;
  const int a0 = turns && !kPairs ? unit * 16 : unit * 32;  // plain units follow the rotated 2 half elements
  const int a1 = turns && !kPairs ? a0 + a.half * 2 : a0 + 16;
  const bool one = a0 < head_bytes, two = a1 < head_bytes;
  float c[8], s[8];
  if (turns && ok) {
    angles4<kAxes>(a, w, unit * 8, c, s);
    angles4<kAxes>(a, w, unit * 8 + 4, c + 4, s + 4);
  }
  {
    const char *const src = a.q + n * a.q_stride;
    char *const dst = a.q_out + n * a.q_out_stride;
    for (int i = part; i < p.q_turns; i += kAtOnce * parts) {
      uint4 x0[kAtOnce], x1[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int head = (i + e * parts) * heads + sub;
        x0[e] = x1[e] = make_uint4(0, 0, 0, 0);
        if (head >= a.q_heads || !ok) continue;  // (a token that is dropped has queries of zeros)
        if (one) x0[e] = ld_stream16(src + head * head_bytes + a0);
        if (two) x1[e] = ld_stream16(src + head * head_bytes + a1);
      }
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) {
        const int head = (i + e * parts) * heads + sub;
        if (head >= a.q_heads) continue;
        if (turns && ok) rotate_unit<T, kPairs>(x0[e], x1[e], c, s);
        if (one) *reinterpret_cast<uint4 *>(dst + head * head_bytes + a0) = x0[e];
        if (two) *reinterpret_cast<uint4 *>(dst + head * head_bytes + a1) = x1[e];
      }
    }
  }
  if (row == nullptr) return;
  float off[8] = {};  // what a turned element may be off, of its pair's sum of magnitudes; position 0 turns nothing, and leaves ties
  if (turns) {
#pragma unroll
    for (int k = 0; k < 8; ++k) off[k] = s[k] == 0.f && fabsf(c[k]) == 1.f ? 0.f : fmaxf(fabsf(c[k]), fabsf(s[k])) * 0x1p-22f;
  }
  for (int i = part - p.k_first + (part < p.k_first ? parts : 0); i < p.k_turns; i += parts) {
    const int head = i * heads + sub;
    if (head >= a.heads - a.q_heads) continue;
    const char *const src = a.k + n * a.k_stride + head * head_bytes;
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (one) x0 = ld_stream16(src + a0);
    if (two) x1 = ld_stream16(src + a1);
    if (p.keys_kept) {
      if (turns) rotate_unit<T, kPairs>(x0, x1, c, s);
      char *const dst = row + a.k_off + head * head_bytes;
      if (one) *reinterpret_cast<uint4 *>(dst + a0) = x0;
      if (two) *reinterpret_cast<uint4 *>(dst + a1) = x1;
      continue;
    }
    float y[16], d[8];  // a thread's first, then its second vector; bounds of the errors of y
    unpack8<T>(x0, y);
    unpack8<T>(x1, y + 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i1 = kPairs ? 2 * k : k, i2 = kPairs ? 2 * k + 1 : k + 8;
      d[k] = 0.f;
      if (turns) {
        const float v1 = y[i1], v2 = y[i2];
        y[i1] = __fmaf_rn(v1, c[k], -__fmul_rn(v2, s[k]));
        y[i2] = __fmaf_rn(v2, c[k], __fmul_rn(v1, s[k]));
        d[k] = (fabsf(v1) + fabsf(v2)) * off[k];
      }
    }
    GroupScale g;
    ExactUnit known;
    uint32_t above[4];
    const bool scaled = quantise_between<kPairs>(y, d, 1 << p.lane_shift, &g, known.bytes, above);
    const bool sure = scaled && known.bytes[0] == above[0] && known.bytes[1] == above[1] && known.bytes[2] == above[2] && known.bytes[3] == above[3];
    known.scale = g.scale;
    if (!all_of(sure, 1 << p.lane_shift)) {
      uint32_t unknown = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) unknown |= differing(known.bytes[e], above[e]) << (4 * e);
      known = exact_unit<T, kPairs, kAxes>(p, w, head, unit, !all_of(scaled, 1 << p.lane_shift), unknown, known);
    }
    char *const dst = row + a.k_off + head * a.key_dim;
    *reinterpret_cast<uint2 *>(dst + (a0 >> 1)) = make_uint2(known.bytes[0], known.bytes[1]);
    *reinterpret_cast<uint2 *>(dst + (a1 >> 1)) = make_uint2(known.bytes[2], known.bytes[3]);
    if (unit == 0) *reinterpret_cast<float *>(row + p.ks_off + head * 4) = known.scale;
  }
  for (int i = part - p.v_first + (part < p.v_first ? parts : 0); i < p.v_turns; i += parts) {
    const int at = i * 32 + lane;
    if (at >= p.value_units) continue;
    const char *const src = a.v + n * a.v_stride + at * 32;
    const uint4 x0 = ld_stream16(src), x1 = ld_stream16(src + 16);
    float y[16], top;
    const bool finite = largest_of16<T>(x0, x1, p.group_threads, &top);
    unpack8<T>(x0, y);
    unpack8<T>(x1, y + 8);
    if (!finite) top = largest_of16(y, p.group_threads);
    const GroupScale g = group_scale(top);
    const uint2 lo = pack8(y, g.inverse), hi = pack8(y + 8, g.inverse);
    *reinterpret_cast<uint4 *>(row + a.v_off + at * 16) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    if ((at & (p.group_threads - 1)) == 0)
      *reinterpret_cast<float *>(row + p.vs_off + (at >> (p.group_threads == 8 ? 3 : 2)) * 4) = g.scale;
  }
}

// What token n says of itself.
template <bool kAxes>
CPKV_DEV Work<kAxes> token_work(const AppendParams &p, int n) {
  Work<kAxes> w;
  w.n = n;
  w.slot = p.slots[n];
  w.pos[0] = p.positions[n];
  if constexpr (kAxes) {
#pragma unroll
    for (int a = 1; a < kMaxAxes; ++a) w.pos[a] = a < p.n_axes ? p.positions[a * p.pos_stride + n] : 0;
  }
  return w;
}

// kAtOnce turns of a token's queries have their loads in flight together: four where it has so
// many, and then five blocks to an SM instead of six.  32 heads of 128 (eight turns): 188 us
// with two and 183 with four for 44600 tokens; 16 heads of 64 (two turns): 163 and 191 us for 131072.
constexpr int append_blocks(int at_once) { return at_once == 4 ? 5 : 6; }

template <typename T, bool kPairs, bool kAxes, int kAtOnce>
__global__ void __launch_bounds__(kAppendThreads, append_blocks(kAtOnce)) append_quantised_kernel(const __grid_constant__ QuantisedParams p) {
  const int64_t jobs = (int64_t)p.a.n_tokens * p.parts.d, step = (int64_t)gridDim.x * (kAppendThreads / 32);
  int64_t job = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  auto token_of = [&](int64_t id) { return id < INT32_MAX ? div_by((int)id, p.parts) : (int)(id / p.parts.d); };
  if (job >= jobs) return;
  Work<kAxes> w = token_work<kAxes>(p.a, token_of(job));
  while (true) {
    const int64_t next = job + step;
    Work<kAxes> then;
    if (next < jobs) then = token_work<kAxes>(p.a, token_of(next));
    quantise_token<T, kPairs, kAxes, kAtOnce>(p, w, (int)(job - (int64_t)w.n * p.parts.d));
    if (next >= jobs) return;
    job = next;
    w = then;
  }
}

template <typename T, int kAtOnce>
auto quantised_kernel(bool pairs, bool axes) {
  if (pairs) return axes ? append_quantised_kernel<T, true, true, kAtOnce> : append_quantised_kernel<T, true, false, kAtOnce>;
  return axes ? append_quantised_kernel<T, false, true, kAtOnce> : append_quantised_kernel<T, false, false, kAtOnce>;
}

template <typename T>
auto quantised_kernel(bool pairs, bool axes, bool many) {
  return many ? quantised_kernel<T, 4>(pairs, axes) : quantised_kernel<T, 2>(pairs, axes);
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
  p.keys_kept = row.keep_keys != 0;
  p.group_threads = value_group(row) / 16;
  p.value_units = row.kv_heads * row.value_dim / 16;
  while (16 << p.lane_shift < row.key_dim) ++p.lane_shift;
  const int heads = 32 >> p.lane_shift;
  p.q_turns = (int)ceil_div(q_heads, heads);
  p.k_turns = (int)ceil_div(row.kv_heads, heads);
  p.v_turns = (int)ceil_div(p.value_units, 32);
  // A warp a token once that gives every SM its warps, shares of tokens before.
  const int64_t turns = p.q_turns + p.k_turns + p.v_turns, warps = (int64_t)device_sm_count() * append_blocks(4) * (kAppendThreads / 32);
  const int parts = (int)std::min<int64_t>(std::max<int64_t>(warps / n_tokens, 1), turns);
  p.parts = fast_div((uint32_t)parts);
  p.k_first = p.q_turns % parts;
  p.v_first = (p.q_turns + p.k_turns) % parts;
  const bool pairs = flags & CPKV_ROTARY_INTERLEAVED, axes = n_axes > 1, many = p.q_turns >= 4;
  auto kernel = dtype == CPKV_BF16 ? quantised_kernel<__nv_bfloat16>(pairs, axes, many) : quantised_kernel<__half>(pairs, axes, many);
  const int grid = persistent_grid((const void *)kernel, kAppendThreads, 0, 16, ceil_div(n_tokens * parts, kAppendThreads / 32));
  return launch_kernel(kernel, dim3(grid), dim3(kAppendThreads), 0, false, (cudaStream_t)stream, p);
}
