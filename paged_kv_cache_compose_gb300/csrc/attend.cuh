// What the attention kernels over paged rows share: the sequences of a call,
// which keys a query sees, and where partial results go.
//
// A sequence is a run of query tokens and the keys they attend to.  Its query
// heads are packed per key/value head: local row R = token * G + g (G query
// heads share one key/value head), so a tile of rows uses each key for all G
// heads.  Query token i of nq stands at position kv_len - nq + i and sees key
// j when j <= position and (position - j < window or j < sinks); without
// `causal` it sees all kv_len keys.
//
// A row's softmax is held as (m, l, o): m the running maximum of
// x = scale * log2(e) * q.k, l = sum 2^(x - m), o = sum 2^(x - m) v, all in 32
// bits; parts over disjoint keys join as
//   m = max m_i, l = sum 2^(m_i - m) l_i, o = sum 2^(m_i - m) o_i.
// A part without keys is m = -inf, l = 0, o = 0.
//
// A product adds weight 0 times the value for a key that a row does not see, which
// is a NaN where that value is infinite or one.  Keys that no query of a sequence
// sees are never read; for those that only some see, the split pass takes infinite
// values out before the product and adds them to the rows that see them (weights are
// positive, so an infinity or a NaN is what they contribute), and the tile pass
// works rows that came out as NaN out again.
#pragma once

#include "paged.cuh"

namespace cpkv {

constexpr float kLog2e = 1.4426950408889634f;

// Weights are rounded to the element type for the product with the values, which is the
// matrix instructions' operand type (their sum is taken before that, in 32 bits): half a
// step of each weight, about as much again as the result's own rounding (bf16 results are
// 0.0017 from those in 64 bits with weights in 32 bits, 0.0018 to 0.0023 so).  fp16 would lose
// weights below 2^-25 whole, so its maximum is held kLift below the scores': weights
// reach up to 2^15 (32768, with the tile pass's threshold of 2^8) and down to 2^-39 of
// the largest, or 2^-32 there.
template <typename T, bool kTile>
constexpr float kLift = std::is_same<T, __half>::value ? (kTile ? 7.f : 15.f) : 0.f;
constexpr float kLn2 = 0.6931471805599453f;

// The requests of a windowed call.
template <int N>
struct Seqs {
  static constexpr int kArray = N;
  const int32_t *kv_lens;  // device lengths, clamped to [0, kv_cap]
  const int32_t *table;    // page ids: row s at s * stride
  int64_t stride;
  int32_t *status;
  int count, uniform_q;  // uniform_q > 0: every sequence has that many query tokens
  int kv_cap;
  int window, sinks;  // window 0: none
  static constexpr int causal = 1;
  int cu_q[N + 1];

  CPKV_DEV int q_begin(int s) const { return uniform_q ? s * uniform_q : cu_q[s]; }
  CPKV_DEV int q_count(int s) const { return uniform_q ? uniform_q : cu_q[s + 1] - cu_q[s]; }
  CPKV_DEV int kv_len(int s) const {
    const int n = kv_lens[s];
    return n < 0 ? 0 : (n > kv_cap ? kv_cap : n);
  }
  CPKV_DEV bool kv_len_bad(int s) const { return kv_lens[s] < 0 || kv_lens[s] > kv_cap; }
  CPKV_DEV const int32_t *pages(int s) const { return table + s * stride; }
  // Sequences with lengths of their own queries; the others have one query each.
  CPKV_DEV int ragged() const { return count; }
  // The sequences that hold a query token, and where it stands in them.
  CPKV_DEV int places(int token, int (&s)[2], int (&i)[2]) const {
    s[0] = uniform_q ? token / uniform_q : upper_index(cu_q, count, token);
    i[0] = token - q_begin(s[0]);
    return 1;
  }
};

// Shared prefixes and suffixes as the sequences of one pass: first the groups
// (every request's query over the prefix), then the requests (one query over its
// own suffix).
template <int N>
struct SharedSeqs {
  static constexpr int kArray = N;
  const int32_t *prefix_pages, *table, *suffix_lens;
  int64_t stride;
  int32_t *status;
  int count, groups, suffix_cap;
  static constexpr int causal = 0, window = 0, sinks = 0;
  int cu_q[N + 1];  // requests before each group
  int kv[N];
  int page0[N];

  CPKV_DEV int q_begin(int s) const { return s < groups ? cu_q[s] : s - groups; }
  CPKV_DEV int q_count(int s) const { return s < groups ? cu_q[s + 1] - cu_q[s] : 1; }
  CPKV_DEV int kv_len(int s) const {
    if (s < groups) return kv[s];
    const int n = suffix_lens[s - groups];
    return n < 0 ? 0 : (n > suffix_cap ? suffix_cap : n);
  }
  CPKV_DEV bool kv_len_bad(int s) const {
    return s >= groups && (suffix_lens[s - groups] < 0 || suffix_lens[s - groups] > suffix_cap);
  }
  CPKV_DEV const int32_t *pages(int s) const {
    return s < groups ? prefix_pages + page0[s] : table + (s - groups) * stride;
  }
  CPKV_DEV int ragged() const { return groups; }
  CPKV_DEV int places(int token, int (&s)[2], int (&i)[2]) const {
    s[0] = groups + token;
    i[0] = 0;
    s[1] = upper_index(cu_q, groups, token);
    i[1] = token - cu_q[s[1]];
    return 2;
  }
};

// Keys that some of the query tokens [i0, i1) of a sequence see, as tiles of
// kTile keys at multiples of kTile: n_sink tiles from key 0 on, then tiles from
// first_tile on.  Keys of those tiles outside [0, sink_end) and [lo, hi) are
// seen by none of them (and never read: their pages may be gone).
struct KeyRange {
  int hi, lo, sink_end;
  int n_sink, first_tile, n_tiles;

  CPKV_DEV int tile_start(int j, int tile) const { return (j < n_sink ? j : first_tile + j - n_sink) * tile; }
  CPKV_DEV bool any_sees(int key) const { return key < sink_end || (key >= lo && key < hi); }
};

template <int kTile>
CPKV_DEV KeyRange key_range(int kv, int nq, int i0, int i1, int causal, int window, int sinks) {
  KeyRange r;
  r.lo = 0;
  r.hi = kv;
  if (causal) {
    const int p0 = kv - nq + i0, p1 = kv - nq + i1 - 1;  // positions of the first and last token
    r.hi = p1 + 1 < 0 ? 0 : p1 + 1;
    if (window > 0 && p0 - window + 1 > 0) r.lo = p0 - window + 1;
  }
  r.sink_end = sinks < r.lo ? sinks : r.lo;
  r.n_sink = (r.sink_end + kTile - 1) / kTile;
  r.first_tile = r.lo / kTile > r.n_sink ? r.lo / kTile : r.n_sink;
  const int end = (r.hi + kTile - 1) / kTile;
  r.n_tiles = r.hi <= 0 ? 0 : r.n_sink + (end > r.first_tile ? end - r.first_tile : 0);
  return r;
}

// One row's visible keys: [lo, hi) and [0, sinks) below hi.
struct RowMask {
  int lo, hi, sinks;
  CPKV_DEV bool sees(int key) const { return key < hi && (key >= lo || key < sinks); }
};

CPKV_DEV RowMask row_mask(int kv, int nq, int i, int causal, int window, int sinks) {
  RowMask m;
  m.lo = 0;
  m.hi = kv;
  m.sinks = sinks;
  if (causal) {
    const int p = kv - nq + i;
    m.hi = p + 1;
    if (window > 0) m.lo = p - window + 1;
  }
  return m;
}

CPKV_DEV float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

CPKV_DEV float log2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A finished row's factor of its output and its log-sum-exp (zeros and -infinity
// where no key had a weight; a NaN stays one).
CPKV_DEV float row_scale(float l) { return l == 0.f ? 0.f : 1.f / l; }
CPKV_DEV float row_lse(float m, float l) { return l == 0.f ? -INFINITY : (m + log2_approx(l)) * kLn2; }

// Where queries come from and results go.
struct AttendIo {
  const char *q;
  char *out;
  float *lse;                    // may be null; [token][q_heads]
  int64_t q_stride, out_stride;  // bytes between tokens
  int q_heads, kv_heads;
  FastDiv group;  // query heads per key/value head
  float scale_log2;
  int64_t k_off, v_off;    // bytes of the keys and values in a row
  int64_t ks_off, vs_off;  // of quantised rows: of the scales
};

// ---------------------------------------------------------------------------
// warp-level matrix instructions on 16-bit operands
// ---------------------------------------------------------------------------
template <typename T>
CPKV_DEV void mma_16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1);
template <>
CPKV_DEV void mma_16816<__nv_bfloat16>(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
CPKV_DEV void mma_16816<__half>(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

CPKV_DEV void ldmatrix_x4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

CPKV_DEV void ldmatrix_x4_trans(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// 16-byte asynchronous copy with an L2 policy; `bytes` 0 writes zeros and reads nothing.
CPKV_DEV void cp_async16_hint(uint32_t smem, const void *src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(smem), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}
CPKV_DEV void cp_async16(uint32_t smem, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}
// Four bytes alike; `bytes` 0 writes zeros and reads nothing.
CPKV_DEV void cp_async4(uint32_t smem, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem), "l"(src), "r"(bytes) : "memory");
}
CPKV_DEV void cp_async16_or_zeros(uint32_t smem, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(src), "r"(bytes) : "memory");
}
CPKV_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
CPKV_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
CPKV_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------------------
// the split pass: parts of sequences of at most 16 packed rows over stretches of keys
// ---------------------------------------------------------------------------
constexpr int kSplitRows = 16;
constexpr int kSplitTile = 64;     // keys of a unit
constexpr int kSplitMaxGrid = 1024;

// Workspace of a split pass over `count` sequences, in order: cum (units of a
// head before each sequence and in all), then the slots' (m, l) pairs, then their values.
// Slots: two per block (its first stretch, and its last when that is another
// sequence's), then one per key/value head and sequence for those that one block holds whole.
struct SplitSpace {
  int32_t *cum;
  float *ml;  // [slot][16][2]
  float *o;   // [slot][16][D]
  int grid;
};

// Units of a cut when a head's `total` are cut into `parts`.
CPKV_DEV int split_chunk(int total, int parts) { return total <= parts ? 1 : (total + parts - 1) / parts; }

template <typename S>
struct SplitParams {
  S seqs;
  PagedPools pools;
  AttendIo io;
  SplitSpace space;
  int direct;  // sequences that one block holds whole go straight to the output
};

// Finds the parts of a row of a split pass.
template <typename S>
struct SplitSource {
  S seqs;
  SplitSpace space;
  int direct;
};

}  // namespace cpkv
