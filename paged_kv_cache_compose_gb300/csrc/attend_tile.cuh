// Attention of many query rows on the tensor core: a block owns 256 packed rows
// of one sequence and key/value head and goes once over the keys they see, 128
// at a time, with the running maximum and sum of each row's softmax.
//
// Two products per 128 keys, 4 * 256 * 128 * D operations on 2 * 128 * D values:
// the tensor core bounds it at D = 128, the exponentials (one per query and key)
// at D = 64.  The 256 rows are two tiles of 128 so that one tile's softmax runs
// while the tensor core multiplies for the other:
//   warps 0..3, 4..7   the softmax of tile 0, 1: a thread owns a row.  Scores come
//                      from tensor memory; weights go back over them, rounded to
//                      the element type (summed before that).
//   warps 8..10        keys and values of the pages to shared memory by cp.async
//                      with a pointer per key, so pages may have any size and
//                      stand in any order.
//   warp 11            issues the products: scores tile by tile (queries, keys in
//                      shared memory), then values (weights in tensor memory).
// Tensor memory (512 columns): scores of the tiles at 0 and 128, outputs at 256
// and 384.  A row's output is rescaled only when its maximum has risen by more
// than 2^8 since the last time: weights stay below 2^8, and the sum and the output
// carry the same factor, which cancels at the end.
#pragma once

#include "attend.cuh"
#include "tcgen05.cuh"

namespace cpkv {

constexpr int kTileRows = 256;  // packed rows of a block
constexpr int kTileKeys = 128;
constexpr int kLoaders = 96;
constexpr int kTileThreads = 256 + kLoaders + 32;
constexpr float kRescaleAt = 8.f;
constexpr uint64_t kTileWaitNs = 2000000000ull;

// Slots of a tile pass: [item][split], an item being (row tile of all
// sequences, key/value head).
struct TileSpace {
  float *ml;  // [slot][256][2]
  float *o;   // [slot][256][D]
  int splits;
};

template <int N>
struct TileParams {
  Seqs<N> seqs;
  PagedPools pools;
  AttendIo io;
  TileSpace space;
  int direct;           // one split, and the rows go straight to the output
  int cu_tiles[N + 1];  // row tiles before each sequence
};

// Finds the parts of a row of a tile pass.
template <int N>
struct TileSource {
  Seqs<N> seqs;
  TileSpace space;
  int cu_tiles[N + 1];
};

template <int D>
struct TileShape {
  static constexpr int kBlocks = D / 64;                     // 64-element blocks of a vector
  static constexpr int kOperand = kTileKeys * D * 2;         // keys (or values, or 128 queries) in shared memory
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQ = 2 * kOperand;
  static constexpr int kPointers = 2 * kTileKeys * 8;
  static constexpr int kSmem = 1024 + kQ + 2 * kStages * kOperand + kPointers;
};

template <int N>
CPKV_DEV int find_tile_seq(const TileParams<N> &p, int tile) {
  return upper_index(p.cu_tiles, p.seqs.count, tile);
}

struct TileBars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], o_full, drain;
  uint32_t tmem;
  int gave_up;
};

// Bounded wait of one thread; false once any warp of the block has given up.
CPKV_DEV bool tile_wait(TileBars *b, uint64_t *bar, uint32_t parity, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int *)&b->gave_up) return false;
    if (global_timer_ns() - t0 > kTileWaitNs) {
      *(volatile int *)&b->gave_up = 1;
      raise_status(status, CPKV_STATUS_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The same for a whole warp, which goes on together.
CPKV_DEV bool tile_wait_warp(TileBars *b, uint64_t *bar, uint32_t parity, int32_t *status) {
  return __all_sync(0xffffffffu, tile_wait(b, bar, parity, status));
}

template <typename T, int D, int N>
__global__ void __launch_bounds__(kTileThreads, 1) attend_tile_kernel(const __grid_constant__ TileParams<N> p) {
  using Shape = TileShape<D>;
  constexpr int kStages = Shape::kStages;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ char raw_smem[];
  __shared__ TileBars bars;
  char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  char *q_smem = smem, *k_smem = smem + Shape::kQ, *v_smem = k_smem + kStages * Shape::kOperand;
  unsigned long long *pointers = reinterpret_cast<unsigned long long *>(v_smem + kStages * Shape::kOperand);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *status = p.seqs.status;

  // this block's item: the last row tiles first, which see the most keys
  const int splits = p.space.splits;
  const int item = (int)(gridDim.x / splits) - 1 - (int)(blockIdx.x / splits);
  const int split = (int)(blockIdx.x % splits);
  const int tile = item / p.io.kv_heads, h = item - tile * p.io.kv_heads;
  const int s = find_tile_seq(p, tile);
  const int rt = tile - p.cu_tiles[s];
  const int group = p.io.group.d, nq = p.seqs.q_count(s), kv = p.seqs.kv_len(s), rows = nq * group;
  const int row0 = rt * kTileRows;
  const int i0 = div_by(row0, p.io.group);
  const int i1 = div_by((row0 + kTileRows < rows ? row0 + kTileRows : rows) - 1, p.io.group) + 1;
  const KeyRange keys = key_range<kTileKeys>(kv, nq, i0, i1, p.seqs.causal, p.seqs.window, p.seqs.sinks);
  const int j0 = (int)((int64_t)keys.n_tiles * split / splits), j1 = (int)((int64_t)keys.n_tiles * (split + 1) / splits);
  const int n = j1 - j0;
  const int tiles = rows - row0 > 128 ? 2 : 1;  // of 128 rows, with any row
  if (threadIdx.x == 0 && split == 0 && h == 0 && rt == 0 && p.seqs.kv_len_bad(s)) raise_status(status, CPKV_STATUS_OUT_CAPACITY);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.k_full[i], kLoaders);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], kLoaders);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t], 128);
    }
    mbar_init(&bars.o_full, 1);
    mbar_init(&bars.drain, 1);
    bars.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 11) tmem_alloc(&bars.tmem, 512);

  // queries: 16-byte chunks, zeros past the last row
  if (n > 0) {
    const int64_t q0 = p.seqs.q_begin(s);
    for (int c = threadIdx.x; c < kTileRows * (D / 8); c += kTileThreads) {
      const int r = c / (D / 8), chunk = c % (D / 8);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row0 + r < rows) {
        const int i = div_by(row0 + r, p.io.group), g = row0 + r - i * group;
        v = ld_stream16(p.io.q + (q0 + i) * p.io.q_stride + ((int64_t)h * group + g) * (D * 2) + chunk * 16);
      }
      const int t = r >> 7, tr = r & 127;
      *reinterpret_cast<uint4 *>(q_smem + t * Shape::kOperand + (chunk >> 3) * (kTileKeys * 128) + tr * 128 +
                                 (((chunk & 7) ^ (tr & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp < 4 * tiles) {
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int row = row0 + (int)threadIdx.x;  // threads 0..127 tile 0, 128..255 tile 1
    const int tile_first = row0 + t * 128;
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) * 32 << 16);
    const uint32_t s_at = lane_base + t * 128, o_at = lane_base + 256 + t * 128;
    const RowMask mask = row_mask(kv, nq, div_by(row, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks);
    int last = tile_first + 127;
    if (last >= rows) last = rows - 1;
    const int full_hi = row_mask(kv, nq, div_by(tile_first, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks).hi;
    const int full_lo = row_mask(kv, nq, div_by(last < 0 ? 0 : last, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks).lo;
    const float scale = p.io.scale_log2;
    float base = -INFINITY, l = 0.f;
    bool ok = true;
    for (int it = 0; it < n; ++it) {
      ok = tile_wait_warp(&bars, &bars.s_full[t], it & 1, status);
      if (!ok) break;
      tmem_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_load32(x[c], s_at + c * 32);
      tmem_wait_loads();
      const int start = keys.tile_start(j0 + it, kTileKeys);
      if (!(start + kTileKeys <= full_hi && (start >= full_lo || start + kTileKeys <= p.seqs.sinks))) {
        const int lo = mask.lo - start, hi = mask.hi - start, sinks = mask.sinks - start;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int j = c * 32 + i;
            if (!(j < hi && (j >= lo || j < sinks))) x[c][i] = 0xff800000u;
          }
      }
      float best[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        best[c] = __uint_as_float(x[c][0]);
#pragma unroll
        for (int i = 1; i < 32; ++i) best[c] = fmaxf(best[c], __uint_as_float(x[c][i]));
      }
      const float top = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])) * scale;
      const bool rise = top > base + kRescaleAt || (base == -INFINITY && top != -INFINITY);
      if (__any_sync(0xffffffffu, rise)) {
        const float next = rise ? top : base;
        const float fall = rise ? exp2_approx(base - next) : 1.f;
        base = next;
        l *= fall;
        if (it > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_load32(o, o_at + c * 32);
            tmem_wait_loads();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fall);
            tmem_store32(o_at + c * 32, o);
          }
        }
      }
      const float shift = base == -INFINITY ? 0.f : base;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = exp2_approx(fmaf(__uint_as_float(x[c][2 * i]), scale, -shift));
          const float b = exp2_approx(fmaf(__uint_as_float(x[c][2 * i + 1]), scale, -shift));
          sum0 += a;
          sum1 += b;
          w[i] = pack2<T>(a, b);
        }
        l += sum0 + sum1;
        tmem_store16(s_at + c * 16, w);
      }
      tmem_wait_stores();
      tmem_fence_before();
      mbar_arrive(&bars.p_full[t]);
    }
    if (ok && n > 0) ok = tile_wait_warp(&bars, &bars.o_full, 0, status);
    tmem_fence_after();
    if (ok && row < rows) {
      const int64_t slot_row = ((int64_t)item * splits + split) * kTileRows + threadIdx.x;
      const int i = div_by(row, p.io.group), head = h * group + row - i * group;
      const int64_t token = p.seqs.q_begin(s) + i;
      if (!p.direct) {
        *reinterpret_cast<float2 *>(p.space.ml + slot_row * 2) = make_float2(base, l);
      } else if (p.io.lse != nullptr) {
        p.io.lse[token * p.io.q_heads + head] = row_lse(base, l);
      }
    }
    if (ok) {
      const float inv = row_scale(l);
      const int64_t slot_row = ((int64_t)item * splits + split) * kTileRows + threadIdx.x;
      const int i = div_by(row, p.io.group), head = h * group + row - i * group;
      char *dst = p.io.out + (p.seqs.q_begin(s) + i) * p.io.out_stride + (int64_t)head * (D * 2);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_load32(o, o_at + c * 32);
          tmem_wait_loads();
        }
        if (row >= rows) continue;
        if (p.direct) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = l == 0.f ? 0u : pack2<T>(__uint_as_float(o[v * 8 + 2 * e]) * inv, __uint_as_float(o[v * 8 + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4 *>(dst + c * 64 + v * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (n > 0) {
          float *to = p.space.o + slot_row * D + c * 32;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *reinterpret_cast<uint4 *>(to + v * 4) = make_uint4(o[v * 4], o[v * 4 + 1], o[v * 4 + 2], o[v * 4 + 3]);
        }
      }
    }
    tmem_fence_before();
  } else if (warp >= 8 && warp < 11) {
    // ---------------------------------------------------------------- loads
    const int lt = (int)threadIdx.x - 256, lw = lt >> 5;
    constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
    const int64_t k_at = p.io.k_off + (int64_t)h * D * 2, v_at = p.io.v_off + (int64_t)h * D * 2;
    const int32_t *pages = p.seqs.pages(s);
    int page[2] = {-1, -1};
    auto look_up = [&](int j) {
      const int start = keys.tile_start(j, kTileKeys);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = lt + e * kLoaders, key = start + r;
        page[e] = -1;
        if (r < kTileKeys && keys.any_sees(key)) page[e] = pages[div_by(key, p.pools.page_size)];
      }
    };
    auto copy = [&](char *to, const unsigned long long *from, int64_t at) {
      const int c = lane % kLanes;
      const uint32_t dst = smem_addr(to) + (c >> 3) * (kTileKeys * 128);
#pragma unroll 4
      for (int g = lw; g < kTileKeys / kRowsAtOnce; g += kLoaders / 32) {
        const int r = g * kRowsAtOnce + lane / kLanes;
        const char *src = reinterpret_cast<const char *>(from[r]);
        const int bytes = src == nullptr ? 0 : 16;
        src = src == nullptr ? p.io.q : src + at + c * 16;
        cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), src, bytes);
      }
      cp_async_commit();
    };
    bool ok = true;
    if (n > 0) look_up(j0);
    int signalled = 0;  // groups whose copies have been announced; group 2 j is keys j, 2 j + 1 values j
    auto announce = [&] {
      fence_proxy_async_smem();
      const int j = signalled >> 1;
      mbar_arrive(signalled & 1 ? &bars.v_full[j % kStages] : &bars.k_full[j % kStages]);
      ++signalled;
    };
    for (int it = 0; it < n; ++it) {
      unsigned long long *mine = pointers + (it & 1) * kTileKeys;
      const int start = keys.tile_start(j0 + it, kTileKeys);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = lt + e * kLoaders, key = start + r;
        if (r >= kTileKeys) continue;
        const char *at = nullptr;
        if (keys.any_sees(key)) {
          at = page_address(p.pools, page[e]);
          if (at == nullptr) {
            raise_status(status, CPKV_STATUS_PAGE_OOB);
          } else {
            at += (int64_t)(key - div_by(key, p.pools.page_size) * (int)p.pools.page_size.d) * p.pools.row_bytes;
          }
        }
        mine[r] = (unsigned long long)at;
      }
      if (it + 1 < n) look_up(j0 + it + 1);
      asm volatile("bar.sync 1, %0;" ::"n"(kLoaders) : "memory");
      const int stage = it % kStages;
      const uint32_t freed = (it / kStages - 1) & 1;
      if (ok && it >= kStages) ok = tile_wait_warp(&bars, &bars.k_empty[stage], freed, status);
      if (!ok) continue;  // the other loading warps still meet at the barrier
      copy(k_smem + stage * Shape::kOperand, mine, k_at);
      if (it >= 1) {
        cp_async_wait<2>();
        announce();
      }
      if (it >= kStages) ok = tile_wait_warp(&bars, &bars.v_empty[stage], freed, status);
      if (!ok) continue;
      copy(v_smem + stage * Shape::kOperand, mine, v_at);
      if (it >= 1) {
        cp_async_wait<2>();
        announce();
      }
    }
    cp_async_wait<0>();
    while (ok && signalled < 2 * n) announce();
  } else if (warp == 11 && n > 0) {
    // ---------------------------------------------------------------- products
    const uint32_t desc_s = product_desc(kBf16, 128, kTileKeys, false), desc_o = product_desc(kBf16, 128, D, true);
    const uint32_t q_addr = smem_addr(q_smem), k_addr = smem_addr(k_smem), v_addr = smem_addr(v_smem);
    auto scores = [&](int t, int it) {
      const uint32_t a = q_addr + t * Shape::kOperand, b = k_addr + (it % kStages) * Shape::kOperand;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = (k >> 2) * (kTileKeys * 128) + (k & 3) * 32;
        mma_ss(tmem + t * 128, operand_desc(a + at, 16), operand_desc(b + at, 16), desc_s, k > 0);
      }
    };
    auto values = [&](int t, int it) {
      const uint32_t b = v_addr + (it % kStages) * Shape::kOperand;
#pragma unroll
      for (int k = 0; k < kTileKeys / 16; ++k)
        mma_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8, operand_desc(b + k * 2048, kTileKeys * 128), desc_o,
               it > 0 || k > 0);
    };
    if (lane == 0) {
      bool ok = tile_wait(&bars, &bars.k_full[0], 0, status);
      if (ok) {
        tmem_fence_after();
        for (int t = 0; t < tiles; ++t) {
          scores(t, 0);
          mma_commit(&bars.s_full[t]);
        }
        mma_commit(&bars.k_empty[0]);
      }
      for (int it = 0; it < n && ok; ++it) {
        const int next = it + 1;
        if (next < n) ok = tile_wait(&bars, &bars.k_full[next % kStages], (next / kStages) & 1, status);
        if (ok) ok = tile_wait(&bars, &bars.v_full[it % kStages], (it / kStages) & 1, status);
        for (int t = 0; t < tiles && ok; ++t) {
          ok = tile_wait(&bars, &bars.p_full[t], it & 1, status);
          if (!ok) break;
          tmem_fence_after();
          values(t, it);
          if (next < n) {
            scores(t, next);
            mma_commit(&bars.s_full[t]);
          }
        }
        if (!ok) break;
        mma_commit(&bars.v_empty[it % kStages]);
        if (next < n) mma_commit(&bars.k_empty[next % kStages]);
      }
      mma_commit(ok ? &bars.o_full : &bars.drain);
      if (!ok) {  // products in flight end before tensor memory is freed
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&bars.drain, 0) && global_timer_ns() - t0 < kTileWaitNs) {
        }
      }
    }
    __syncwarp();
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 11) tmem_free(tmem, 512);
}

}  // namespace cpkv
