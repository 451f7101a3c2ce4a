// Joins the parts of each row: m = max m_i, l = sum 2^(m_i - m) l_i,
// o = sum 2^(m_i - m) o_i, out = o / l.
#pragma once

#include "attend_split.cuh"
#include "attend_tile.cuh"

namespace cpkv {

// Parts of one row within a pass: rows `first`, then `next`, next + step, ... of
// its (m, l) pairs and values.
struct Parts {
  const float *ml, *o;
  int64_t first, next, step;
  int count;
  CPKV_DEV int64_t row(int k) const { return k == 0 ? first : next + (k - 1) * step; }
};

// Where a pass keeps a query row: found from the call's own inputs, before the
// pass has ended.
struct Spot {
  int s, rt, in_tile, n_tiles;
};

template <typename S>
CPKV_DEV Spot find_spot(const SplitSource<S> &src, const AttendIo &io, int s, int i, int g) {
  const int nq = src.seqs.q_count(s);
  const KeyRange keys = key_range<kSplitTile>(src.seqs.kv_len(s), nq, 0, nq, src.seqs.causal, src.seqs.window, src.seqs.sinks);
  return Spot{s, 0, i * (int)io.group.d + g, keys.n_tiles};
}

template <typename S>
CPKV_DEV Spot find_spot(const TileSource<S> &src, const AttendIo &io, int s, int i, int g) {
  const int row = i * (int)io.group.d + g;
  return Spot{s, row / kTileRows, row % kTileRows, 0};
}

// The parts of a row of key/value head h; false when the pass has written that
// row's output itself.
template <typename S>
CPKV_DEV bool find_parts(Parts *r, const SplitSource<S> &src, const AttendIo &io, const Spot &at, int h) {
  r->ml = src.space.ml;
  r->o = src.space.o;
  r->count = 0;
  if (at.n_tiles == 0) return true;
  const int chunk = split_chunk(src.space.cum[src.seqs.count], src.space.grid / io.kv_heads);
  const int begin = src.space.cum[at.s], end = begin + at.n_tiles;
  const int c0 = begin / chunk, c1 = (end - 1) / chunk;
  r->count = c1 - c0 + 1;
  if (c0 == c1) {
    if (src.direct) return false;
    const int64_t slot = 2 * (int64_t)src.space.grid + (int64_t)h * src.seqs.count + at.s;
    r->first = slot * kSplitRows + at.in_tile;
    return true;
  }
  // the sequence's stretch is the last of cut c0 unless it begins there, and the first of the others
  const int64_t slot = 2 * ((int64_t)c0 * io.kv_heads + h);
  r->first = (slot + (begin == c0 * chunk ? 0 : 1)) * kSplitRows + at.in_tile;
  r->step = 2 * (int64_t)io.kv_heads * kSplitRows;
  r->next = slot * kSplitRows + r->step + at.in_tile;
  return true;
}

template <typename S>
CPKV_DEV bool find_parts(Parts *r, const TileSource<S> &src, const AttendIo &io, const Spot &at, int h) {
  const TileSpace &space = src.space;
  r->ml = space.ml;
  r->o = space.o;
  if (at.s < src.seqs.ragged()) {
    const int64_t item = (int64_t)(src.cu_tiles[at.s] + at.rt) * io.kv_heads + h;
    r->count = space.splits;
    r->step = kTileRows;
    r->first = item * space.splits * kTileRows + at.in_tile;
  } else {
    const int64_t item = ((int64_t)(at.s - src.seqs.ragged()) * io.kv_heads + h) * space.single_tiles + at.rt;
    r->count = space.single_splits;
    r->step = single_rows(io.group.d);
    r->first = space.single_row + item * space.single_splits * r->step + at.in_tile;
  }
  r->next = r->first + r->step;
  return true;
}

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

template <typename Source>
struct JoinParams {
  Source source;
  AttendIo io;
  int64_t rows;  // tokens * q_heads
};

// kWarps warps per row (token, query head), four rows or one to a block.  Each
// lane takes one part of a batch of 32: its maximum and sum, then its weight and
// address, which go round as the warps add the parts' values, every kWarps-th one
// each.  Latency bounds it (a few hundred to some thousand rows, a chain of three
// reads from L2), so one batch holds a row's parts of prefix and suffix.
template <typename T, int D, typename Source, int kWarps>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ JoinParams<Source> p) {
  constexpr int kEach = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part_of = kWarps == 1 ? 0 : warp;
  const int64_t row = kWarps == 1 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;
  if (row >= p.rows) return;
  const int token = (int)(row / p.io.q_heads), head = (int)(row - (int64_t)token * p.io.q_heads);
  const int h = div_by(head, p.io.group), g = head - h * (int)p.io.group.d;
  const Spots spots = find_spots(p.source, p.io, token, g);
  wait_prerequisite();
  Parts parts[2] = {};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k < spots.count && !find_parts(&parts[k], p.source, p.io, spots.at[k], h)) return;
  const int c0 = parts[0].count, count = c0 + parts[1].count;

  float m = -INFINITY, l = 0.f, o[kEach] = {};
  for (int k0 = 0; k0 < count; k0 += 32) {
    const int k = k0 + lane;
    float2 v = make_float2(-INFINITY, 0.f);
    const float *values = nullptr;
    if (k < count) {
      const Parts &at = k < c0 ? parts[0] : parts[1];
      const int64_t r = at.row(k < c0 ? k : k - c0);
      v = *reinterpret_cast<const float2 *>(at.ml + r * 2);
      if (v.y != 0.f) values = at.o + r * D;  // a part without keys has no values written
    }
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
#pragma unroll 8
    for (int i = part_of; i < n; i += kWarps) {
      const float w = __shfl_sync(0xffffffffu, weight, i);
      const float *src = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, (unsigned long long)values, i));
      if (src == nullptr) continue;  // (a weight of 0 still lets infinite values through, as in one pass)
      src += lane * kEach;
      if constexpr (kEach == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(src);
        o[0] += w * x.x, o[1] += w * x.y, o[2] += w * x.z, o[3] += w * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2 *>(src);
        o[0] += w * x.x, o[1] += w * x.y;
      }
    }
  }
  if constexpr (kWarps > 1) {
    __shared__ float others[kWarps - 1][D];
    if (warp > 0) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) others[warp - 1][lane * kEach + e] = o[e];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
#pragma unroll
      for (int e = 0; e < kEach; ++e) o[e] += others[w][lane * kEach + e];
  }
  const float inv = row_scale(l);
  char *dst = p.io.out + token * p.io.out_stride + (int64_t)head * D * 2 + lane * (D / 16);
  if constexpr (D == 128) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv));
  } else {
    *reinterpret_cast<uint32_t *>(dst) = pack2<T>(o[0] * inv, o[1] * inv);
  }
  if (p.io.lse != nullptr && lane == 0) p.io.lse[row] = row_lse(m, l);
}

}  // namespace cpkv
