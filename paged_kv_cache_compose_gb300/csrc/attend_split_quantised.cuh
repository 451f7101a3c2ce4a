// The split pass over quantised rows: stretches of the line of units, as in
// attend_split.cuh, with half the bytes a key.
//
// The matrix instructions take fp16, which holds every e4m3 number, so keys and
// values go into them as they are kept and the scales stay outside the products:
//   x_ij = (scale log2(e) a_i s_j) (q_i / a_i . k_j),
// s_j the key's scale and a_i a power of two that brings the largest element of a
// bf16 query to [2^14, 2^15) (fp16 queries are taken as they are, a_i = 1): of its other
// elements only the parts below 2^-39 of that one round.  The values' scales t_j go into
// the weights,
//   o_i = sum_j 2^(x_ij + log2 t_j - n_i) v_j,   l_i = sum_j 2^(x_ij - m_i),
// with a reference n_i of their own, so that neither a row of zeros (t_j = 2^-126) nor a
// large one costs the other weights their bits.  m_i and n_i follow the largest exponents with a
// little slack (kSlackQ).  One conversion a pair of elements and a second exponential a score:
// with e4m3 * scale in the element type it were five instructions a pair.
//
// Keys and values are the first operand, of 16 keys (or 16 elements) by 16, and the queries
// (the weights) the second, 8 rows at a time: a key converted once serves 8 rows, or 16 with
// a second product, and what a lane holds of outputs, queries and scores halves for the 8
// rows or fewer that a decode step of most models has.  A lane's four bytes of a 16-byte
// chunk c of a key are elements 16 c + 4 t .. + 3 (t = lane % 4), so the queries' fragments hold
// those; values come by transposed pairs of bytes, sorted into two columns of keys by one
// permutation, so a lane's outputs are elements 16 c + 2 g and + 1 (g = lane / 4) of rows 2 t and + 1.
//
// Measured with the joining pass: 64 requests of 8 query rows, 8 heads of 64, the last 4096 of up
// to 65536 keys, 66.7 us (4.2 TB/s; instructions issue in 60% of the cycles), 96.7 with queries and
// weights as the first operand and 16 rows always; 12 requests of 12 query rows on 8 heads of 128,
// up to 16384 keys in one-token pages, 67.8 us (3.8 TB/s).  A unit at a time, with half the
// loads in flight and a vote for each: 77 and 73 us.
#pragma once

#include "attend_split.cuh"
#include "quantised.cuh"

namespace cpkv {

// kBlocks8 8 rows at a time: 1 or 2.
template <int D, SplitMode kMode, int kBlocks8>
struct SplitShapeQ {
  static constexpr int kUnits = 2;                         // units that a warp takes at once
  static constexpr int kKeys = kUnits * kWarpKeys;         // its keys of them
  static constexpr int kVectors = 2 * kKeys * D;           // keys, then values
  static constexpr int kStage = kVectors + 2 * kKeys * 4;  // then their scales
  static constexpr int kStages = kMode == kFewKeys ? 3 : 2;
  // Blocks to an SM: as many as registers and two stages in shared memory allow.
  static constexpr int kBlocks = kMode == kFewKeys ? 1 : kBlocks8 == 1 ? (D == 128 ? 3 : 5) : (D == 128 ? 2 : 3);
  static constexpr int kRing = kSplitWarps * kStages * kStage;
  static constexpr int kJoin = 8 * kBlocks8 * D * 4;  // half the columns of two warps while a sequence's parts are joined
  static constexpr int kSmem = kRing + kJoin + kSplitWarps * kSplitRows * 8;
};

// The weights' maximum is held kLiftQ below the scores', and let go kSlackQ above itself before
// anything is rescaled (most units end there, after one vote): weights reach 2^15 in fp16 and
// are held to half a step of 2^-24, 2^-37 of the largest.
constexpr float kLiftQ = 12.f, kSlackQ = 3.f;

// Bytes 0, 2, 1, 3.
CPKV_DEV uint32_t sort_pairs(uint32_t v) { return __byte_perm(v, 0, 0x3120); }

// The 8 x 8 matrix of fp16 whose rows the warp's lanes hold four to one, the other way round.
CPKV_DEV uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The factor that brings a query of this largest magnitude (the bits of a bf16 number) to
// [2^14, 2^15), and its inverse.
CPKV_DEV float2 query_factors(uint32_t largest) {
  const int e = max((int)(largest >> 7) & 0xff, 15);  // at most 254 + 15: both are normal numbers
  return make_float2(__uint_as_float((uint32_t)min(268 - e, 254) << 23), __uint_as_float((uint32_t)max(e - 14, 1) << 23));
}

template <typename T, int D, typename S, SplitMode kMode, int kBlocks8>
__global__ void __launch_bounds__(kSplitWarps * 32, SplitShapeQ<D, kMode, kBlocks8>::kBlocks) attend_split_quantised_kernel(const __grid_constant__ SplitParams<S> p) {
  using Shape = SplitShapeQ<D, kMode, kBlocks8>;
  using P = SplitParams<S>;
  constexpr bool kWhole = kMode != kLine;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int kChunks = D / 16;  // 16-byte chunks of a vector
  constexpr int kUnits = Shape::kUnits, kKeys = Shape::kKeys;
  extern __shared__ __align__(128) char smem[];
  __shared__ int scan_scratch[33];
  __shared__ int few_pages[kWhole ? kSplitWarps : 1][kWholeUnits][kWarpKeys];
  int *cum = reinterpret_cast<int *>(smem + Shape::kSmem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  release_dependents();  // the joining kernel, which waits for this one
  const int head = (int)blockIdx.x % p.io.kv_heads;  // key/value head
  Cursor<P> ld;
  int u0, u1;
  if (!find_stretch<kMode>(p, head, cum, scan_scratch, &ld, &u0, &u1)) return;

  char *ring = smem + warp * Shape::kStages * Shape::kStage;
  const uint32_t ring_addr = smem_addr(ring);
  float *join = reinterpret_cast<float *>(smem + Shape::kRing);
  float2 *ml = reinterpret_cast<float2 *>(smem + Shape::kRing + Shape::kJoin);
  // where chunk c of a key lies: eight neighbouring keys' in different banks
  auto place = [](int key, int c) { return key * D + ((c ^ (D == 128 ? key & 7 : key >> 1 & 3)) << 4); };

  // Loads: lanes 0..15 own a key each of one unit, the others of the next, which is taken with it
  // where it is of the same sequence.
  const uint64_t once = l2_policy_evict_first();
  Cursor<P> at = ld;
  auto together = [&](const Cursor<P> &c, int u) { return min(min(kUnits, c.units - c.j), u1 - u); };
  const int sub = lane >> 4;
  int ld_u = u0, ld_key = 0, ld_page = -1;
  bool ld_sees = false;
  auto look_up = [&] {  // the page of this lane's key, one turn ahead of its copy
    ld_key = ld.keys.tile_start(ld.j + sub, kSplitTile) + warp * kWarpKeys + (lane & 15);
    ld_sees = sub < together(ld, ld_u) && ld.keys.any_sees(ld_key);
    if (kWhole && ld.j + sub < kWholeUnits) {
      ld_page = few_pages[warp][ld.j + sub][lane & 15];
    } else {
      ld_page = ld_sees ? p.seqs.pages(ld.s)[div_by(ld_key, p.pools.page_size)] : -1;
    }
  };
  if constexpr (kWhole) {  // all page ids of the sequence at once: one latency, not one per unit
#pragma unroll
    for (int i = 0; i < kWholeUnits; i += 2) {
      const int j = i + (lane >> 4), key = ld.keys.tile_start(j, kSplitTile) + warp * kWarpKeys + (lane & 15);
      if (j < u1 && ld.keys.any_sees(key)) few_pages[warp][j][lane & 15] = p.seqs.pages(ld.s)[div_by(key, p.pools.page_size)];
    }
    __syncwarp();
  }
  if (u0 < u1) look_up();
  auto load_next = [&](int stage) {
    if (ld_u < u1) {
      const char *row = nullptr;
      if (ld_sees) {
        row = page_address(p.pools, ld_page);
        if (row == nullptr) {
          raise_status(p.seqs.status, CPKV_STATUS_PAGE_OOB);
        } else {
          row += (int64_t)(ld_key - div_by(ld_key, p.pools.page_size) * (int)p.pools.page_size.d) * p.pools.row_bytes;
        }
      }
      constexpr int kRows = 32 / kChunks;  // keys of one warp-wide copy
      const int c = lane % kChunks;
      const uint32_t dst = ring_addr + stage * Shape::kStage;
      const char *const none = reinterpret_cast<const char *>(p.io.q);  // a valid address that is not read
      const int64_t k_at = p.io.k_off + (int64_t)head * D + c * 16;
      const int64_t v_at = p.io.v_off + (int64_t)head * D + c * 16;
      const char *const scales_at = row == nullptr ? none : row + (int64_t)head * 4;
      cp_async4(dst + Shape::kVectors + lane * 4, row == nullptr ? none : scales_at + p.io.ks_off, row == nullptr ? 0 : 4);
      cp_async4(dst + Shape::kVectors + (kKeys + lane) * 4, row == nullptr ? none : scales_at + p.io.vs_off, row == nullptr ? 0 : 4);
#pragma unroll
      for (int i = 0; i < kKeys / kRows; ++i) {
        const int key = i * kRows + lane / kChunks;
        const char *src = reinterpret_cast<const char *>(__shfl_sync(0xffffffffu, (unsigned long long)row, key));
        const int bytes = src == nullptr ? 0 : 16;
        const uint32_t to = dst + place(key, c);
        cp_async16_hint(to, bytes ? src + k_at : none, bytes, once);
        cp_async16_hint(to + kKeys * D, bytes ? src + v_at : none, bytes, once);
      }
      const int taken = together(ld, ld_u);
      ld_u += taken;
      if (ld_u < u1) {
        ld.j += taken - 1;
        ld.advance(p);
        look_up();
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < Shape::kStages - 1; ++i) load_next(i);

  int stage = 0, seg_j0 = 0;
  bool fresh = true, first_segment = true;
  const int t = lane & 3, g = lane >> 2;  // this lane's rows are 2 t and 2 t + 1 of each 8, its keys g and g + 8
  uint32_t qf[kBlocks8][kChunks][2];
  float o[kBlocks8][kChunks][4];  // of chunk c: element 2 g of both rows, then 2 g + 1
  float m[kBlocks8][2], l[kBlocks8][2], n[kBlocks8][2];  // references of the weights' exponents and their sum; of the weights times the values' scales
  float factor[kBlocks8][2];                             // of the products of a row
  RowMask mask[kBlocks8][2];
  int full_lo = 0, full_hi = 0;  // keys in [full_lo, full_hi) are seen by every row

  // A sequence's rows from here on.
  auto begin_rows = [&] {
    seg_j0 = at.j;
    const int group = p.io.group.d, rows = at.nq * group;
    const int q0 = p.seqs.q_begin(at.s);
    full_hi = row_mask(at.kv, at.nq, 0, p.seqs.causal, p.seqs.window, p.seqs.sinks).hi;
    full_lo = row_mask(at.kv, at.nq, at.nq - 1, p.seqs.causal, p.seqs.window, p.seqs.sinks).lo;
#pragma unroll
    for (int b = 0; b < kBlocks8; ++b) {
      const int row = 8 * b + g;
      const bool in = row < rows;
      const int i = div_by(row, p.io.group), h = row - i * group;
      const char *src = p.io.q + (q0 + i) * p.io.q_stride + ((int64_t)head * group + h) * (D * 2) + t * 8;
      uint32_t largest = 0;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint2 v = in ? *reinterpret_cast<const uint2 *>(src + c * 32) : make_uint2(0u, 0u);
        qf[b][c][0] = v.x;
        qf[b][c][1] = v.y;
        if constexpr (!kHalf) largest = __vmaxu2(largest, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
      }
      float mine = p.io.scale_log2;
      if constexpr (!kHalf) {
        largest = max(largest & 0xffffu, largest >> 16);
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        const float2 f = query_factors(largest);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 v = unpack2<__nv_bfloat16>(qf[b][c][e]);
            qf[b][c][e] = pack2<__half>(v.x * f.x, v.y * f.x);
          }
        mine *= f.y;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        factor[b][r] = __shfl_sync(0xffffffffu, mine, (2 * t + r) * 4);
        mask[b][r] = row_mask(at.kv, at.nq, div_by(8 * b + 2 * t + r, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks);
        m[b][r] = n[b][r] = -INFINITY;
        l[b][r] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][c][e] = 0.f;
    }
  };
  // The end of a sequence or of this block's stretch of it: `complete` when the block held it whole.
  auto end_rows = [&](bool complete) {
    // join the four warps' parts: common reference, then values pairwise
#pragma unroll
    for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[b][r] += __shfl_xor_sync(0xffffffffu, l[b][r], w);
        if (g == 0) ml[warp * kSplitRows + 8 * b + 2 * t + r] = make_float2(m[b][r], l[b][r]);
      }
    __syncthreads();
    float big[kBlocks8][2], sum[kBlocks8][2];
#pragma unroll
    for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float2 v[kSplitWarps];
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) {
          v[w] = ml[w * kSplitRows + 8 * b + 2 * t + r];
          top = fmaxf(top, v[w].x);
        }
        const float base = top == -INFINITY ? 0.f : top;
        big[b][r] = top;
        sum[b][r] = 0.f;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) sum[b][r] += exp2_approx(v[w].x - base) * v[w].y;
        // the values' scales come back here, in two factors: 2^-126 and less (scales below some 2^-112) would be flushed to 0
        const float to = n[b][r] - base, by = fmaxf(to, -100.f), mine = exp2_approx(by), rest = exp2_approx(to - by);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          o[b][c][r] = o[b][c][r] * mine * rest;
          o[b][c][2 + r] = o[b][c][2 + r] * mine * rest;
        }
      }
    auto each = [&](int columns, float *buf, bool put) {
#pragma unroll
      for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
        for (int c = 0; c < kChunks / 2; ++c) {
          float4 *q = reinterpret_cast<float4 *>(buf) + (b * (kChunks / 2) + c) * 32 + lane;
          float *mine = o[b][columns * (kChunks / 2) + c];
          if (put) {
            *q = make_float4(mine[0], mine[1], mine[2], mine[3]);
          } else {
            const float4 v = *q;
            mine[0] += v.x, mine[1] += v.y, mine[2] += v.z, mine[3] += v.w;
          }
        }
    };
    float *const upper = join + 8 * kBlocks8 * D / 2;
#pragma unroll
    for (int columns = 0; columns < 2; ++columns) {
      if (warp >= 2) each(columns, warp == 2 ? join : upper, true);
      __syncthreads();
      if (warp < 2) each(columns, warp == 0 ? join : upper, false);
      if (warp == 1) each(columns, upper, true);
      __syncthreads();
      if (warp == 0) each(columns, upper, false);
      __syncthreads();
    }
    if (warp == 0) {
      const int group = p.io.group.d, rows = at.nq * group;
      const int64_t slot = complete ? 2 * (int64_t)gridDim.x + (int64_t)head * p.seqs.count + at.s
                                    : 2 * (int64_t)blockIdx.x + (first_segment ? 0 : 1);
#pragma unroll
      for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 8 * b + 2 * t + r;
          if (row >= rows) continue;
          if (complete && p.direct) {
            const int i = div_by(row, p.io.group);
            const int64_t token = p.seqs.q_begin(at.s) + i;
            const int q_head = head * group + row - i * group;
            const float inv = row_scale(sum[b][r]);
            char *dst = p.io.out + token * p.io.out_stride + (int64_t)q_head * (D * 2) + g * 4;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              *reinterpret_cast<uint32_t *>(dst + c * 32) = pack2<T>(o[b][c][r] * inv, o[b][c][2 + r] * inv);
            if (p.io.lse != nullptr && g == 0) p.io.lse[token * p.io.q_heads + q_head] = row_lse(big[b][r], sum[b][r]);
          } else {
            float *dst = p.space.o + (slot * kSplitRows + row) * D + g * 2;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) *reinterpret_cast<float2 *>(dst + c * 16) = make_float2(o[b][c][r], o[b][c][2 + r]);
            if (g == 0) *reinterpret_cast<float2 *>(p.space.ml + (slot * kSplitRows + row) * 2) = make_float2(big[b][r], sum[b][r]);
          }
        }
    }
  };

  if constexpr (kWhole) begin_rows();
  for (int u = u0, taken; u < u1; u += taken) {
    if (!kWhole && fresh) {
      fresh = false;
      begin_rows();
    }
    taken = together(at, u);
    cp_async_wait<Shape::kStages - 2>();
    __syncwarp();
    load_next(stage == 0 ? Shape::kStages - 1 : stage - 1);

    // products of this warp's 16 keys of each unit and the rows
    const uint32_t kb = ring_addr + stage * Shape::kStage;
    const float *const scales = reinterpret_cast<const float *>(ring + stage * Shape::kStage + Shape::kVectors);
    float x[kBlocks8][kUnits][4] = {};  // rows 2 t, 2 t + 1 of key g, then of key g + 8
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int key = 16 * i + (lane & 15);
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t v[4];
        ldmatrix_x4(v, kb + place(key, c + (lane >> 4)));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t a[4] = {halves_low(v[2 * e]), halves_low(v[2 * e + 1]), halves_high(v[2 * e]), halves_high(v[2 * e + 1])};
#pragma unroll
          for (int b = 0; b < kBlocks8; ++b) mma_16816<__half>(x[b][i], a, qf[b][c + e][0], qf[b][c + e][1]);
        }
      }
    }
    float y[kBlocks8][kUnits][4];  // with the values' scales
    bool whole = true;             // every row sees all keys
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int key0 = at.keys.tile_start(at.j + i, kSplitTile) + warp * kWarpKeys;
      const bool all = i < taken && key0 + kWarpKeys <= full_hi && (key0 >= full_lo || key0 + kWarpKeys <= p.seqs.sinks);
      const float ks[2] = {scales[16 * i + g], scales[16 * i + g + 8]};
      const float lift[2] = {log2_approx(scales[kKeys + 16 * i + g]), log2_approx(scales[kKeys + 16 * i + g + 8])};
#pragma unroll
      for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e & 1, k = e >> 1;
          x[b][i][e] *= factor[b][r] * ks[k];
          y[b][i][e] = x[b][i][e] + lift[k];
          if (!all && !(i < taken && mask[b][r].sees(key0 + g + 8 * k))) x[b][i][e] = y[b][i][e] = -INFINITY;
        }
      whole &= all;
    }
    bool rise = false;
    float best[kBlocks8][2], top[kBlocks8][2];
#pragma unroll
    for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[b][r] = fmaxf(fmaxf(x[b][0][r], x[b][0][2 + r]), fmaxf(x[b][1][r], x[b][1][2 + r]));
        top[b][r] = fmaxf(fmaxf(y[b][0][r], y[b][0][2 + r]), fmaxf(y[b][1][r], y[b][1][2 + r]));
        rise |= best[b][r] - m[b][r] > kSlackQ || top[b][r] - n[b][r] > kLiftQ + kSlackQ;
      }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) {
            best[b][r] = fmaxf(best[b][r], __shfl_xor_sync(0xffffffffu, best[b][r], w));
            top[b][r] = fmaxf(top[b][r], __shfl_xor_sync(0xffffffffu, top[b][r], w));
          }
          const float next = fmaxf(m[b][r], best[b][r]), up = fmaxf(n[b][r], top[b][r] - kLiftQ);
          l[b][r] *= exp2_approx(m[b][r] - (next == -INFINITY ? 0.f : next));
          const float fall = exp2_approx(n[b][r] - (up == -INFINITY ? 0.f : up));
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            o[b][c][r] *= fall;
            o[b][c][2 + r] *= fall;
          }
          m[b][r] = next;
          n[b][r] = up;
        }
    }
    uint32_t pf[kBlocks8][kUnits][2];  // weights as the second operand; rounded to fp16 for the product, summed before it
#pragma unroll
    for (int b = 0; b < kBlocks8; ++b) {
      const float shift[2] = {m[b][0] == -INFINITY ? 0.f : m[b][0], m[b][1] == -INFINITY ? 0.f : m[b][1]};
      const float over[2] = {n[b][0] == -INFINITY ? 0.f : n[b][0], n[b][1] == -INFINITY ? 0.f : n[b][1]};
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[b][e & 1] += exp2_approx(x[b][i][e] - shift[e & 1]);
          w[e] = exp2_approx(y[b][i][e] - over[e & 1]);
        }
        pf[b][i][0] = transposed(pack2<__half>(w[0], w[1]));
        pf[b][i][1] = transposed(pack2<__half>(w[2], w[3]));
      }
    }
    if (S::causal && !whole && at.nq > 1) {  // values that are no numbers, of keys that some rows do not see
      char *const values = ring + stage * Shape::kStage + kKeys * D;
      uint32_t marks = 0;
#pragma unroll
      for (int i = 0; i < kKeys * D / 512; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(values)[i * 32 + lane];
        marks |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) | ((v.z & 0x7f7f7f7fu) + 0x01010101u) |
                 ((v.w & 0x7f7f7f7fu) + 0x01010101u);
      }
      if (__any_sync(0xffffffffu, (marks & 0x80808080u) != 0)) {
        for (int key = 0; key < 16 * taken; ++key) {
          const int number = at.keys.tile_start(at.j + key / 16, kSplitTile) + warp * kWarpKeys + key % 16;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const uint32_t v = *reinterpret_cast<const uint16_t *>(values + place(key, c) + g * 2);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if ((v >> (8 * e) & 0x7f) == 0x7f) {
#pragma unroll
                for (int b = 0; b < kBlocks8; ++b)
#pragma unroll
                  for (int r = 0; r < 2; ++r)
                    if (mask[b][r].sees(number)) o[b][c][2 * e + r] = NAN;
              }
          }
        }
        __syncwarp();
        for (int i = lane; i < kKeys * D / 4; i += 32) {
          uint32_t *const v = reinterpret_cast<uint32_t *>(values) + i;
          *v &= ~((((*v & 0x7f7f7f7fu) + 0x01010101u & 0x80808080u) >> 7) * 0xffu);
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int key = 16 * i + (lane & 15);
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t v[4];  // keys 0..7 and 8..15 of chunk c, then of the next
        ldmatrix_x4_trans(v, kb + kKeys * D + place(key, c + (lane >> 4)));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t lo = sort_pairs(v[2 * e]), hi = sort_pairs(v[2 * e + 1]);
          const uint32_t a[4] = {halves_low(lo), halves_high(lo), halves_low(hi), halves_high(hi)};
#pragma unroll
          for (int b = 0; b < kBlocks8; ++b) mma_16816<__half>(o[b][c + e], a, pf[b][i][0], pf[b][i][1]);
        }
      }
    }
    __syncwarp();
    stage = stage + 1 == Shape::kStages ? 0 : stage + 1;

    const bool keys_end = at.j + taken == at.units;
    if (kWhole || (!keys_end && u + taken < u1)) {
      at.j += taken;
      continue;
    }
    end_rows(keys_end && seg_j0 == 0);

    first_segment = false;
    fresh = true;
    if (u + taken < u1) {
      at.j += taken - 1;
      at.advance(p);
    }
  }
  cp_async_wait<0>();
  if constexpr (kWhole) end_rows(true);
  if (!kWhole && blockIdx.x == gridDim.x - 1) wait_prerequisite();  // the joining kernel waits for this one only
}

}  // namespace cpkv
