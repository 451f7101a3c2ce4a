// Joins the parts of each row: m = max m_i, l = sum 2^(m_i - m) l_i,
// o = sum 2^(m_i - m) o_i, out = o / l.
#pragma once

#include "attend_split.cuh"
#include "attend_tile.cuh"

namespace cpkv {

// One row on its way: m, l and this lane's D / 32 elements of o.
template <int D>
struct RowSum {
  static constexpr int kEach = D / 32;
  float m = -INFINITY, l = 0.f, o[kEach] = {};

  // `count` parts; `at(k)` is part k's row in (m, l) pairs `ml` and values `ov`.
  template <typename F>
  CPKV_DEV void add(const float *ml, const float *ov, int count, int lane, F at) {
    for (int k0 = 0; k0 < count; k0 += 32) {
      float2 v = make_float2(-INFINITY, 0.f);
      if (k0 + lane < count) v = *reinterpret_cast<const float2 *>(ml + at(k0 + lane) * 2);
      float best = v.x;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, w));
      const float next = fmaxf(m, best), base = next == -INFINITY ? 0.f : next;
      const float fall = exp2_approx(m - base), weight = exp2_approx(v.x - base);
      float sum = weight * v.y;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l = l * fall + sum;
      m = next;
#pragma unroll
      for (int e = 0; e < kEach; ++e) o[e] *= fall;
      const int n = count - k0 < 32 ? count - k0 : 32;
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float w = __shfl_sync(0xffffffffu, weight, i);
        if (w == 0.f) continue;  // a part without keys has no values written
        const float *src = ov + at(k0 + i) * D + lane * kEach;
        if constexpr (kEach == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(src);
          o[0] += w * x.x, o[1] += w * x.y, o[2] += w * x.z, o[3] += w * x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(src);
          o[0] += w * x.x, o[1] += w * x.y;
        }
      }
    }
  }
};

// Where a pass keeps a query row: found from the call's own inputs, before the
// pass has ended.
struct Spot {
  int s, rt, in_tile, n_tiles;
};

template <typename S>
CPKV_DEV Spot find_spot(const SplitSource<S> &src, const AttendIo &io, int s, int i, int g) {
  const int nq = src.seqs.q_count(s), row = i * (int)io.group.d + g;
  const KeyRange keys = key_range<kSplitTile>(src.seqs.kv_len(s), nq, 0, nq, src.seqs.causal, src.seqs.window, src.seqs.sinks);
  return Spot{s, row / kSplitRows, row % kSplitRows, keys.n_tiles};
}

template <int N>
CPKV_DEV Spot find_spot(const TileSource<N> &src, const AttendIo &io, int s, int i, int g) {
  const int row = i * (int)io.group.d + g;
  return Spot{s, row / kTileRows, row % kTileRows, 0};
}

// Adds the parts of a row of key/value head h; false when the pass has written
// that row's output itself.
template <int D, typename S>
CPKV_DEV bool add_parts(RowSum<D> *sum, const SplitSource<S> &src, const AttendIo &io, const Spot &at, int h, int lane) {
  if (at.n_tiles == 0) return true;
  const int chunk = split_chunk(src.space.cum[src.seqs.count], src.space.grid / io.kv_heads);
  const int begin = src.space.cum[at.s] + at.rt * at.n_tiles, end = begin + at.n_tiles;
  const int c0 = begin / chunk, c1 = (end - 1) / chunk;
  if (c0 == c1) {
    if (src.direct) return false;
    const int64_t slot = 2 * (int64_t)src.space.grid + h * src.tiles_cap + src.seqs.tiles_before(at.s, io.group.d) + at.rt;
    sum->add(src.space.ml, src.space.o, 1, lane, [&](int) { return slot * kSplitRows + at.in_tile; });
    return true;
  }
  // the tile's stretch is the last of cut c0 unless it begins there, and the first of the others
  const int late = begin == c0 * chunk ? 0 : 1;
  sum->add(src.space.ml, src.space.o, c1 - c0 + 1, lane, [&](int k) {
    return (2 * ((int64_t)(c0 + k) * io.kv_heads + h) + (k == 0 ? late : 0)) * kSplitRows + at.in_tile;
  });
  return true;
}

template <int D, int N>
CPKV_DEV bool add_parts(RowSum<D> *sum, const TileSource<N> &src, const AttendIo &io, const Spot &at, int h, int lane) {
  const int64_t item = (int64_t)(src.cu_tiles[at.s] + at.rt) * io.kv_heads + h;
  const int64_t first = item * src.space.splits * kTileRows + at.in_tile;
  sum->add(src.space.ml, src.space.o, src.space.splits, lane, [&](int k) { return first + (int64_t)k * kTileRows; });
  return true;
}

struct NoSource {};

// The places of a query row in a pass.
struct Spots {
  Spot at[2];
  int count;
};

template <typename Source>
CPKV_DEV Spots find_spots(const Source &src, const AttendIo &io, int token, int g) {
  int s[2], i[2];
  Spots r;
  r.count = src.seqs.places(token, s, i);
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < r.count) r.at[k] = find_spot(src, io, s[k], i[k], g);
  return r;
}

// All parts of a row that a pass has; false when the pass wrote the row itself.
template <int D, typename Source>
CPKV_DEV bool add_all(RowSum<D> *sum, const Source &src, const AttendIo &io, const Spots &spots, int h, int lane) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < spots.count && !add_parts(sum, src, io, spots.at[k], h, lane)) return false;
  return true;
}

// `a`: a pass over the query tokens; `b`: a second one over the same, or none.
template <typename A, typename B>
struct JoinParams {
  A a;
  B b;
  AttendIo io;
  int64_t rows;  // tokens * q_heads
};

// A warp per row (token, query head).
template <typename T, int D, typename A, typename B>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ JoinParams<A, B> p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const int token = (int)(row / p.io.q_heads), head = (int)(row - (int64_t)token * p.io.q_heads);
  const int h = div_by(head, p.io.group), g = head - h * (int)p.io.group.d;
  const Spots a = find_spots(p.a, p.io, token, g);
  Spots b;
  if constexpr (!std::is_same<B, NoSource>::value) b = find_spots(p.b, p.io, token, g);
  wait_prerequisite();
  RowSum<D> sum;
  if (!add_all(&sum, p.a, p.io, a, h, lane)) return;
  if constexpr (!std::is_same<B, NoSource>::value) add_all(&sum, p.b, p.io, b, h, lane);
  const float inv = row_scale(sum.l);
  char *dst = p.io.out + token * p.io.out_stride + (int64_t)head * D * 2 + lane * (D / 16);
  if constexpr (D == 128) {
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(pack2<T>(sum.o[0] * inv, sum.o[1] * inv), pack2<T>(sum.o[2] * inv, sum.o[3] * inv));
  } else {
    *reinterpret_cast<uint32_t *>(dst) = pack2<T>(sum.o[0] * inv, sum.o[1] * inv);
  }
  if (p.io.lse != nullptr && lane == 0) p.io.lse[row] = row_lse(sum.m, sum.l);
}

}  // namespace cpkv
