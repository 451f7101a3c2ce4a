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
// with a maximum n_i of their own, so that neither a row of zeros (t_j = 2^-126) nor a
// large one costs the other weights their bits.  One conversion a pair of elements and a
// second exponential a score: with e4m3 * scale in the element type it were five
// instructions a pair.
//
// Fragments: a lane's four bytes of a 16-byte chunk c of a key are elements
// 16 c + 4 t .. + 3 (t = lane % 4), so the queries' fragments hold those; values come
// by transposed pairs of bytes, sorted into two columns of keys by one permutation, so
// a lane's outputs are elements 16 c + 4 t .. + 3 of its rows too.
#pragma once

#include "attend_split.cuh"
#include "quantised.cuh"

namespace cpkv {

template <int D, SplitMode kMode>
struct SplitShapeQ {
  static constexpr int kVectors = 2 * kWarpKeys * D;               // keys, then values
  static constexpr int kStage = kVectors + 2 * kWarpKeys * 4;      // then their scales
  static constexpr int kStages = kMode == kFewKeys ? 5 : 4;
  static constexpr int kBlocks = kMode == kFewKeys ? 1 : D == 128 ? 3 : 5;  // blocks to an SM
  static constexpr int kRing = kSplitWarps * kStages * kStage;
  static constexpr int kJoin = kSplitRows * D * 4;  // half the columns of two warps while a sequence's parts are joined
  static constexpr int kSmem = kRing + kJoin + kSplitWarps * kSplitRows * 8;
};

// Bytes 0, 2, 1, 3.
CPKV_DEV uint32_t sort_pairs(uint32_t v) { return __byte_perm(v, 0, 0x3120); }

// The factor that brings a query of this largest magnitude (the bits of a bf16 number) to
// [2^14, 2^15), and its inverse.
CPKV_DEV float2 query_factors(uint32_t largest) {
  const int e = max((int)(largest >> 7) & 0xff, 15);  // at most 254 + 15: both are normal numbers
  return make_float2(__uint_as_float((uint32_t)min(268 - e, 254) << 23), __uint_as_float((uint32_t)max(e - 14, 1) << 23));
}

template <typename T, int D, typename S, SplitMode kMode>
__global__ void __launch_bounds__(kSplitWarps * 32, SplitShapeQ<D, kMode>::kBlocks) attend_split_quantised_kernel(const __grid_constant__ SplitParams<S> p) {
  using Shape = SplitShapeQ<D, kMode>;
  using P = SplitParams<S>;
  constexpr bool kWhole = kMode != kLine;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int kChunks = D / 16;  // 16-byte chunks of a vector
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

  // loads: lanes 0..15 own one key each, as in the other split pass
  const uint64_t once = l2_policy_evict_first();
  Cursor<P> at = ld;
  int ld_u = u0, ld_key = 0, ld_page = -1;
  bool ld_sees = false;
  auto look_up = [&] {  // the page of this lane's key, one unit ahead of its copy
    ld_key = ld.keys.tile_start(ld.j, kSplitTile) + warp * kWarpKeys + (lane & 15);
    ld_sees = ld.keys.any_sees(ld_key);
    if (kWhole && ld.j < kWholeUnits) {
      ld_page = few_pages[warp][ld.j][lane & 15];
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
      const int64_t s_at = (lane < 16 ? p.io.ks_off : p.io.vs_off) + (int64_t)head * 4;
      cp_async4(dst + Shape::kVectors + lane * 4, row == nullptr ? none : row + s_at, row == nullptr ? 0 : 4);
#pragma unroll
      for (int i = 0; i < kWarpKeys / kRows; ++i) {
        const int key = i * kRows + lane / kChunks;
        const char *src = reinterpret_cast<const char *>(__shfl_sync(0xffffffffu, (unsigned long long)row, key));
        const int bytes = src == nullptr ? 0 : 16;
        const uint32_t to = dst + place(key, c);
        cp_async16_hint(to, bytes ? src + k_at : none, bytes, once);
        cp_async16_hint(to + kWarpKeys * D, bytes ? src + v_at : none, bytes, once);
      }
      if (++ld_u < u1) {
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
  uint32_t qf[kChunks][4];
  float o[kChunks][2][4];  // of chunk c: elements 4 t, 4 t + 2 and 4 t + 1, 4 t + 3 of both rows
  float m[2], l[2], n[2];  // maximum and sum of the weights; maximum of the weights times the values' scales
  float factor[2];         // of the products of a row
  RowMask mask[2];
  int full_lo = 0, full_hi = 0;  // keys in [full_lo, full_hi) are seen by every row

  // A sequence's rows from here on.
  auto begin_rows = [&] {
    seg_j0 = at.j;
    const int group = p.io.group.d, rows = at.nq * group;
    const int q0 = p.seqs.q_begin(at.s);
    full_hi = row_mask(at.kv, at.nq, 0, p.seqs.causal, p.seqs.window, p.seqs.sinks).hi;
    full_lo = row_mask(at.kv, at.nq, at.nq - 1, p.seqs.causal, p.seqs.window, p.seqs.sinks).lo;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = (lane >> 2) + 8 * r;
      const bool in = row < rows;
      const int i = div_by(row, p.io.group), g = row - i * group;
      mask[r] = row_mask(at.kv, at.nq, i, p.seqs.causal, p.seqs.window, p.seqs.sinks);
      const char *src = p.io.q + (q0 + i) * p.io.q_stride + ((int64_t)head * group + g) * (D * 2) + (lane & 3) * 8;
      uint32_t largest = 0;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint2 v = in ? *reinterpret_cast<const uint2 *>(src + c * 32) : make_uint2(0u, 0u);
        qf[c][r] = v.x;
        qf[c][r + 2] = v.y;
        if constexpr (!kHalf) largest = __vmaxu2(largest, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
      }
      factor[r] = p.io.scale_log2;
      if constexpr (!kHalf) {
        largest = max(largest & 0xffffu, largest >> 16);
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        const float2 f = query_factors(largest);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int h = 0; h < 4; h += 2) {
            const float2 v = unpack2<__nv_bfloat16>(qf[c][r + h]);
            qf[c][r + h] = pack2<__half>(v.x * f.x, v.y * f.x);
          }
        factor[r] *= f.y;
      }
      m[r] = n[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[c][i >> 2][i & 3] = 0.f;
  };
  // The end of a sequence or of this block's stretch of it: `complete` when the block held it whole.
  auto end_rows = [&](bool complete) {
    // join the four warps' parts: common maximum, then values pairwise
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) ml[warp * kSplitRows + (lane >> 2) + 8 * r] = make_float2(m[r], l[r]);
    }
    __syncthreads();
    float big[2], sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = (lane >> 2) + 8 * r;
      float2 v[kSplitWarps];
      big[r] = -INFINITY;
#pragma unroll
      for (int w = 0; w < kSplitWarps; ++w) {
        v[w] = ml[w * kSplitRows + row];
        big[r] = fmaxf(big[r], v[w].x);
      }
      const float base = big[r] == -INFINITY ? 0.f : big[r];
      sum[r] = 0.f;
#pragma unroll
      for (int w = 0; w < kSplitWarps; ++w) sum[r] += exp2_approx(v[w].x - base) * v[w].y;
      const float mine = exp2_approx(n[r] - base);  // the values' scales come back here
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[c][h][2 * r] *= mine;
          o[c][h][2 * r + 1] *= mine;
        }
    }
    auto each = [&](int columns, float *buf, bool put) {
#pragma unroll
      for (int c = 0; c < kChunks / 2; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 *q = reinterpret_cast<float4 *>(buf) + (2 * c + h) * 32 + lane;
          float *mine = o[columns * (kChunks / 2) + c][h];
          if (put) {
            *q = make_float4(mine[0], mine[1], mine[2], mine[3]);
          } else {
            const float4 v = *q;
            mine[0] += v.x, mine[1] += v.y, mine[2] += v.z, mine[3] += v.w;
          }
        }
    };
    float *const upper = join + kSplitRows * D / 2;
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
      for (int r = 0; r < 2; ++r) {
        const int row = (lane >> 2) + 8 * r;
        if (row >= rows) continue;
        if (complete && p.direct) {
          const int i = div_by(row, p.io.group), g = row - i * group;
          const int64_t token = p.seqs.q_begin(at.s) + i;
          const int q_head = head * group + g;
          const float inv = row_scale(sum[r]);
          char *dst = p.io.out + token * p.io.out_stride + (int64_t)q_head * (D * 2) + (lane & 3) * 8;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            *reinterpret_cast<uint2 *>(dst + c * 32) = make_uint2(pack2<T>(o[c][0][2 * r] * inv, o[c][1][2 * r] * inv),
                                                                 pack2<T>(o[c][0][2 * r + 1] * inv, o[c][1][2 * r + 1] * inv));
          if (p.io.lse != nullptr && (lane & 3) == 0)
            p.io.lse[token * p.io.q_heads + q_head] = row_lse(big[r], sum[r]);
        } else {
          float *dst = p.space.o + (slot * kSplitRows + row) * D + (lane & 3) * 4;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            *reinterpret_cast<float4 *>(dst + c * 16) = make_float4(o[c][0][2 * r], o[c][1][2 * r], o[c][0][2 * r + 1], o[c][1][2 * r + 1]);
          if ((lane & 3) == 0)
            *reinterpret_cast<float2 *>(p.space.ml + (slot * kSplitRows + row) * 2) = make_float2(big[r], sum[r]);
        }
      }
    }
  };

  if constexpr (kWhole) begin_rows();
  for (int u = u0; u < u1; ++u) {
    if (!kWhole && fresh) {
      fresh = false;
      begin_rows();
    }
    cp_async_wait<Shape::kStages - 2>();
    __syncwarp();
    load_next(stage == 0 ? Shape::kStages - 1 : stage - 1);

    // products of 16 rows and this warp's 16 keys
    const uint32_t kb = ring_addr + stage * Shape::kStage;
    const float *const scales = reinterpret_cast<const float *>(ring + stage * Shape::kStage + Shape::kVectors);
    float x[2][4] = {};
    {
      const int key = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t b[4];
        ldmatrix_x4(b, kb + place(key, c + ((lane >> 3) & 1)));
        mma_16816<__half>(x[0], qf[c], halves_low(b[0]), halves_high(b[0]));
        mma_16816<__half>(x[1], qf[c], halves_low(b[2]), halves_high(b[2]));
        mma_16816<__half>(x[0], qf[c + 1], halves_low(b[1]), halves_high(b[1]));
        mma_16816<__half>(x[1], qf[c + 1], halves_low(b[3]), halves_high(b[3]));
      }
    }
    const int key0 = at.keys.tile_start(at.j, kSplitTile) + warp * kWarpKeys;
    const bool whole = key0 + kWarpKeys <= full_hi && (key0 >= full_lo || key0 + kWarpKeys <= p.seqs.sinks);
    float y[2][4];  // with the values' scales
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 ks = *reinterpret_cast<const float2 *>(scales + e * 8 + (lane & 3) * 2);
      const float2 vs = *reinterpret_cast<const float2 *>(scales + kWarpKeys + e * 8 + (lane & 3) * 2);
      const float lift[2] = {log2_approx(vs.x), log2_approx(vs.y)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[e][i] *= factor[i >> 1] * (i & 1 ? ks.y : ks.x);
        y[e][i] = x[e][i] + lift[i & 1];
        if (!whole && !mask[i >> 1].sees(key0 + e * 8 + (lane & 3) * 2 + (i & 1))) x[e][i] = y[e][i] = -INFINITY;
      }
    }
    uint32_t pf[4];  // weights as the first operand; rounded to fp16 for the product, summed before it
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float best = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
      float top = fmaxf(fmaxf(y[0][2 * r], y[0][2 * r + 1]), fmaxf(y[1][2 * r], y[1][2 * r + 1]));
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float next = fmaxf(m[r], best), up = fmaxf(n[r], top - kLift<__half, false>);
      const float shift = next == -INFINITY ? 0.f : next, over = up == -INFINITY ? 0.f : up;
      l[r] *= exp2_approx(m[r] - shift);
      const float fall = exp2_approx(n[r] - over);
      if (__any_sync(0xffffffffu, up != n[r])) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            o[c][h][2 * r] *= fall;
            o[c][h][2 * r + 1] *= fall;
          }
      }
      m[r] = next;
      n[r] = up;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[r] += exp2_approx(x[e][2 * r] - shift) + exp2_approx(x[e][2 * r + 1] - shift);
        pf[2 * e + r] = pack2<__half>(exp2_approx(y[e][2 * r] - over), exp2_approx(y[e][2 * r + 1] - over));
      }
    }
    if (S::causal && !whole && at.nq > 1) {  // values that are no numbers, of keys that some rows do not see
      char *const values = ring + stage * Shape::kStage + kWarpKeys * D;
      uint32_t marks = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(values)[i * 32 + lane];
        marks |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) | ((v.z & 0x7f7f7f7fu) + 0x01010101u) |
                 ((v.w & 0x7f7f7f7fu) + 0x01010101u);
      }
      if (__any_sync(0xffffffffu, (marks & 0x80808080u) != 0)) {
        for (int key = 0; key < kWarpKeys; ++key) {
          const bool sees[2] = {mask[0].sees(key0 + key), mask[1].sees(key0 + key)};
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(values + place(key, c) + (lane & 3) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((v >> (8 * i) & 0x7f) == 0x7f) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  if (sees[r]) o[c][i & 1][2 * r + (i >> 1)] = NAN;
              }
          }
        }
        __syncwarp();
        for (int i = lane; i < kWarpKeys * D / 4; i += 32) {
          uint32_t *const v = reinterpret_cast<uint32_t *>(values) + i;
          *v &= ~((((*v & 0x7f7f7f7fu) + 0x01010101u & 0x80808080u) >> 7) * 0xffu);
        }
        __syncwarp();
      }
    }
    {
      const int key = lane & 15;
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        uint32_t b[4];
        ldmatrix_x4_trans(b, kb + kWarpKeys * D + place(key, c + (lane >> 4)));
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = sort_pairs(b[i]);
        mma_16816<__half>(o[c][0], pf, halves_low(b[0]), halves_low(b[1]));
        mma_16816<__half>(o[c][1], pf, halves_high(b[0]), halves_high(b[1]));
        mma_16816<__half>(o[c + 1][0], pf, halves_low(b[2]), halves_low(b[3]));
        mma_16816<__half>(o[c + 1][1], pf, halves_high(b[2]), halves_high(b[3]));
      }
    }
    __syncwarp();
    stage = stage + 1 == Shape::kStages ? 0 : stage + 1;

    const bool keys_end = at.j + 1 == at.units;
    if (kWhole || (!keys_end && u + 1 < u1)) {
      ++at.j;
      continue;
    }
    end_rows(keys_end && seg_j0 == 0);

    first_segment = false;
    fresh = true;
    if (u + 1 < u1) at.advance(p);
  }
  cp_async_wait<0>();
  if constexpr (kWhole) end_rows(true);
}

}  // namespace cpkv
