// Attention of few query rows (at most 16 packed ones a sequence) over long paged keys: the keys are cut into
// stretches, each block reduces its stretch to (m, l, o), and a second kernel
// joins the parts of each row.
//
// Bytes bound it: 16 packed rows do 4 D * 16 operations on the 4 D bytes of a
// key and its value, far below what the matrix instructions give, so what
// counts is bytes in flight.  Work is counted in units of 64 keys of one
// sequence; all units of a key/value head form one line that is cut
// evenly over the head's blocks, whatever the lengths are, and a block's warps each
// own 16 keys of every unit with a cp.async ring of their own, so that no block-wide
// barrier stands inside a stretch.  The lines of all heads are cut alike and
// neighbouring blocks hold the same stretch of different heads: a token's heads lie
// side by side in its row, and read together they cost DRAM one page opening
// (64 requests of 4100 keys, 8 heads of 64: 120 us when a block's stretch ran from
// one head into the next, 106 us so).  Warps, not stages, hide the rest: two stages
// and as many blocks as registers allow take 100 us, four stages and three blocks 106.
// With rows that make room in L2 first and the join's set-up beside this pass the
// same step takes 88 us, 5.9 TB/s and 89% of the measured copy rate.  Where every
// sequence has few keys a block takes one whole sequence instead and nothing is left to join.
#pragma once

#include "attend.cuh"

namespace cpkv {

constexpr int kSplitWarps = 4;
constexpr int kWarpKeys = kSplitTile / kSplitWarps;  // 16

// How a block finds its work: a stretch of the line of units, or one sequence of few keys
// (with a deeper ring: its time is that of a few loads).
enum SplitMode { kLine, kFewKeys };
constexpr int kWholeUnits = 8;  // most units of a sequence of few keys

template <int D, SplitMode kMode>
struct SplitShape {
  static constexpr int kRow = D * 2;                       // bytes of a key (or value) vector
  static constexpr int kStage = kWarpKeys * kRow * 2;      // keys, then values
  static constexpr int kStages = kMode == kFewKeys ? 5 : 2;
  static constexpr int kBlocks = kMode == kFewKeys ? 1 : D == 128 ? 3 : 5;  // blocks to an SM
  static constexpr int kRing = kSplitWarps * kStages * kStage;
  static constexpr int kJoin = kSplitRows * D * 4;         // half the columns of two warps while a sequence's parts are joined
  static constexpr int kSmem = kRing + kJoin + kSplitWarps * kSplitRows * 8;
};

// A position on the line of units.
template <typename P>
struct Cursor {
  int s, j, units;
  int nq, kv;
  KeyRange keys;

  CPKV_DEV void enter(const P &p, int seq) {
    s = seq;
    nq = p.seqs.q_count(s);
    kv = p.seqs.kv_len(s);
    keys = key_range<kSplitTile>(kv, nq, 0, nq, p.seqs.causal, p.seqs.window, p.seqs.sinks);
    units = nq > 0 ? keys.n_tiles : 0;
  }
  CPKV_DEV void seek(const P &p, const int *cum, int u) {
    enter(p, upper_index(cum, p.seqs.count, u));
    j = u - cum[s];
  }
  // To the next unit of the line; there must be one.
  CPKV_DEV void advance(const P &p) {
    if (++j < units) return;
    j = 0;
    do {
      enter(p, s + 1);
    } while (units == 0);
  }
};

// This block's units [u0, u1) and a cursor at the first; false where there is none for it.
template <SplitMode kMode, typename P>
CPKV_DEV bool find_stretch(const P &p, int head, int *cum, int *scan_scratch, Cursor<P> *ld, int *u0, int *u1) {
  const int count = p.seqs.count;
  if constexpr (kMode != kLine) {
    ld->enter(p, (int)blockIdx.x / p.io.kv_heads);
    ld->j = 0;
    if (head == 0 && threadIdx.x == 0 && p.seqs.kv_len_bad(ld->s))
      raise_status(p.seqs.status, CPKV_STATUS_OUT_CAPACITY);
    *u0 = 0;
    *u1 = ld->keys.n_tiles;
  } else {
    // units before each sequence
    int total = 0;
    for (int s0 = 0; s0 < count; s0 += kSplitWarps * 32) {
      const int s = s0 + (int)threadIdx.x;
      int mine = 0;
      if (s < count) {
        Cursor<P> c;
        c.enter(p, s);
        mine = c.units;
        if (blockIdx.x == 0 && p.seqs.kv_len_bad(s)) raise_status(p.seqs.status, CPKV_STATUS_OUT_CAPACITY);
      }
      int part;
      const int before = block_exclusive_scan(mine, scan_scratch, &part);
      if (s < count) {
        cum[s] = total + before;
        if (blockIdx.x == 0) p.space.cum[s] = total + before;
      }
      total += part;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.space.cum[count] = total;
    __syncthreads();
    const int chunk = split_chunk(total, (int)gridDim.x / p.io.kv_heads);
    const int64_t first = (int64_t)((int)blockIdx.x / p.io.kv_heads) * chunk;
    if (first >= total) {
      wait_prerequisite();
      return false;
    }
    *u0 = (int)first;
    *u1 = (int)min64(first + chunk, total);
    ld->seek(p, cum, *u0);
  }
  return true;
}

template <typename T, int D, typename S, SplitMode kMode>
__global__ void __launch_bounds__(kSplitWarps * 32, SplitShape<D, kMode>::kBlocks) attend_split_kernel(const __grid_constant__ SplitParams<S> p) {
  using Shape = SplitShape<D, kMode>;
  using P = SplitParams<S>;
  constexpr bool kWhole = kMode != kLine;
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

  // loads: lanes 0..15 own one key each.  A row is read once, by its head's packed
  // rows: it makes room in L2 before the parts do.
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
      constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a vector, keys of one warp-wide copy
      const int c = lane % kLanes;
      const uint32_t dst = ring_addr + stage * Shape::kStage;
      const int64_t k_at = p.io.k_off + (int64_t)head * Shape::kRow + c * 16;
      const int64_t v_at = p.io.v_off + (int64_t)head * Shape::kRow + c * 16;
#pragma unroll
      for (int i = 0; i < kWarpKeys / kRows; ++i) {
        const int key = i * kRows + lane / kLanes;
        const char *src = reinterpret_cast<const char *>(__shfl_sync(0xffffffffu, (unsigned long long)row, key));
        const int bytes = src == nullptr ? 0 : 16;
        if (src == nullptr) src = reinterpret_cast<const char *>(p.io.q);  // a valid address that is not read
        const uint32_t to = dst + key * Shape::kRow + ((c ^ (key & 7)) << 4);
        cp_async16_hint(to, bytes ? src + k_at : src, bytes, once);
        cp_async16_hint(to + kWarpKeys * Shape::kRow, bytes ? src + v_at : src, bytes, once);
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
  uint32_t qf[D / 16][4];
  float o[D / 8][4], m[2], l[2];
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
      const char *src = p.io.q + (q0 + i) * p.io.q_stride + ((int64_t)head * group + g) * Shape::kRow + (lane & 3) * 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][r] = in ? *reinterpret_cast<const uint32_t *>(src + k * 32) : 0u;
        qf[k][r + 2] = in ? *reinterpret_cast<const uint32_t *>(src + k * 32 + 16) : 0u;
      }
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
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
      const float mine = exp2_approx(m[r] - base);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * r] *= mine;
        o[n][2 * r + 1] *= mine;
      }
    }
    auto each = [&](int columns, float *buf, bool put) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float2 *q = reinterpret_cast<float2 *>(buf + (n * 32 + lane) * 4 + 2 * r);
          float *mine = o[columns * (D / 16) + n] + 2 * r;
          if (put) {
            *q = make_float2(mine[0], mine[1]);
          } else {
            mine[0] += q->x;
            mine[1] += q->y;
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
          char *dst = p.io.out + token * p.io.out_stride + (int64_t)q_head * Shape::kRow + (lane & 3) * 4;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<uint32_t *>(dst + n * 16) = pack2<T>(o[n][2 * r] * inv, o[n][2 * r + 1] * inv);
          if (p.io.lse != nullptr && (lane & 3) == 0)
            p.io.lse[token * p.io.q_heads + q_head] = row_lse(big[r], sum[r]);
        } else {
          float *dst = p.space.o + (slot * kSplitRows + row) * D + (lane & 3) * 2;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
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

    // x = scale log2(e) q.k of 16 rows and this warp's 16 keys
    const uint32_t kb = ring_addr + stage * Shape::kStage;
    float x[2][4] = {};
    {
      const int key = (lane & 7) + ((lane >> 4) << 3);
      const uint32_t row = kb + key * Shape::kRow;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldmatrix_x4(b, row + (((2 * k + ((lane >> 3) & 1)) ^ (key & 7)) << 4));
        mma_16816<T>(x[0], qf[k], b[0], b[1]);
        mma_16816<T>(x[1], qf[k], b[2], b[3]);
      }
    }
    const int key0 = at.keys.tile_start(at.j, kSplitTile) + warp * kWarpKeys;
    const bool whole = key0 + kWarpKeys <= full_hi && (key0 >= full_lo || key0 + kWarpKeys <= p.seqs.sinks);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[n][i] *= p.io.scale_log2;
        if (!whole && !mask[i >> 1].sees(key0 + n * 8 + (lane & 3) * 2 + (i & 1))) x[n][i] = -INFINITY;
      }
    float shift[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float best = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
      const float next = fmaxf(m[r], best - kLift<T, false>);
      shift[r] = next == -INFINITY ? 0.f : next;
      const float fall = exp2_approx(m[r] - shift[r]);
      if (__any_sync(0xffffffffu, next != m[r])) {
        l[r] *= fall;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          o[n][2 * r] *= fall;
          o[n][2 * r + 1] *= fall;
        }
      }
      m[r] = next;
    }
    uint32_t pf[4];  // weights as the first operand; rounded to T for the product, summed before it (kLift says why)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float a = exp2_approx(x[n][2 * r] - shift[r]), b = exp2_approx(x[n][2 * r + 1] - shift[r]);
        l[r] += a + b;
        pf[2 * n + r] = pack2<T>(a, b);
      }
    if (S::causal && !whole && at.nq > 1) {  // infinite values of keys that some rows do not see
      char *const values = ring + stage * Shape::kStage + kWarpKeys * Shape::kRow;
      uint4 marks = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) marks = mark_infinite<T>(reinterpret_cast<const uint4 *>(values)[i * 32 + lane], marks);
      if (__any_sync(0xffffffffu, (marks.x | marks.y | marks.z | marks.w) != 0)) {
        for (int key = 0; key < kWarpKeys; ++key) {
          const bool sees[2] = {mask[0].sees(key0 + key), mask[1].sees(key0 + key)};
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const float2 v = unpack2<T>(infinite_of<T>(
                *reinterpret_cast<const uint32_t *>(values + key * Shape::kRow + ((n ^ (key & 7)) << 4) + (lane & 3) * 4)));
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (sees[r]) o[n][2 * r] += v.x, o[n][2 * r + 1] += v.y;
          }
        }
        __syncwarp();
        for (int i = lane; i < kWarpKeys * Shape::kRow / 4; i += 32) {
          uint32_t *const v = reinterpret_cast<uint32_t *>(values) + i;
          *v = finite_of<T>(*v);
        }
        __syncwarp();
      }
    }
    {
      const int key = lane & 15;
      const uint32_t row = kb + kWarpKeys * Shape::kRow + key * Shape::kRow;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldmatrix_x4_trans(b, row + (((2 * n + (lane >> 4)) ^ (key & 7)) << 4));
        mma_16816<T>(o[2 * n], pf, b[0], b[1]);
        mma_16816<T>(o[2 * n + 1], pf, b[2], b[3]);
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
