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
//   warps 8..11        keys and values of the pages to shared memory, 32 keys each:
//                      as TMA boxes where a page holds 16 rows or more and all 32
//                      keys are there, else by cp.async with an address per key, so
//                      pages may have any size and stand in any order.
//   warp 12            issues the products: scores (queries, keys in shared memory),
//                      then values (weights in tensor memory), tile by tile.
// Weights are handed over in two halves of 64 keys: the first half's product runs
// while the second half's exponentials do.
// Tensor memory (512 columns): scores of the tiles at 0 and 128, outputs at 256
// and 384.  A row's output is rescaled only when its maximum has risen by more
// than 2^8 since the last time: weights stay below 2^8, and the sum and the output
// carry the same factor, which cancels at the end.
#pragma once

#include <cuda.h>

#include "attend.cuh"
#include "tcgen05.cuh"

namespace cpkv {

constexpr int kTileRows = 256;  // packed rows of a block
constexpr int kTileKeys = 128;
constexpr int kLoaders = 128;
constexpr int kTileThreads = 512;
// Registers a thread: 512 threads are launched with 128 each, 65536 in all; the
// softmax holds a row's 128 scores.  256 * 192 + 256 * 64 = 65536.
constexpr int kSoftmaxRegisters = 192, kOtherRegisters = 64;
constexpr int kTileMaps = 8;  // most pools that TMA maps travel for
constexpr float kRescaleAt = 8.f;
constexpr uint64_t kTileWaitNs = 2000000000ull;
constexpr uint32_t kTileParkNs = 500000;

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
  int box_rows;         // rows of a TMA box (32 or 16); 0: no maps
  int cu_tiles[N + 1];  // row tiles before each sequence
  CUtensorMap maps[kTileMaps];  // pool r as [rows][elements], boxes of box_rows x 64
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
  static constexpr int kOperand = kTileKeys * D * 2;  // keys (or values, or 128 queries) in shared memory
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQ = 2 * kOperand;
  static constexpr int kSmem = 1024 + kQ + 2 * kStages * kOperand;
};

template <int N>
CPKV_DEV int find_tile_seq(const TileParams<N> &p, int tile) {
  return upper_index(p.cu_tiles, p.seqs.count, tile);
}

struct TileBars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2][2], o_full[2], q_full;
  uint32_t tmem;
  int gave_up;
};

__device__ const uint4 zero_row[16] = {};  // a key or value vector of zeros

// Bounded wait of one thread; false once any warp of the block has given up.
// The hardware parks the thread until the phase ends or the hint (0.5 ms) has passed.
CPKV_DEV bool tile_wait(TileBars *b, uint64_t *bar, uint32_t parity, int32_t *status) {
  if (mbar_try_wait_for(bar, parity, kTileParkNs)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait_for(bar, parity, kTileParkNs)) {
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
  __shared__ ulonglong2 addresses[kTileKeys];  // of the keys being copied: key, value
  char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  char *q_smem = smem, *k_smem = smem + Shape::kQ, *v_smem = k_smem + kStages * Shape::kOperand;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *status = p.seqs.status;
  release_dependents();  // later passes of the call; the joining kernel waits for this one

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

  if (threadIdx.x == 0) {
    if (split == 0 && h == 0 && rt == 0 && p.seqs.kv_len_bad(s)) raise_status(status, CPKV_STATUS_OUT_CAPACITY);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.k_full[i], kLoaders);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], kLoaders);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.o_full[t], 1);
      mbar_init(&bars.p_full[t][0], 128);
      mbar_init(&bars.p_full[t][1], 128);
    }
    mbar_init(&bars.q_full, 256);
    bars.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&bars.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp < 8) {
    // ---------------------------------------------------------------- queries, softmax
    grow_registers<kSoftmaxRegisters>();
    if (n > 0) {  // a warp's threads copy 32 / (D / 8) rows at a time
      constexpr int kLanes = D / 8;
      const int c = threadIdx.x % kLanes;
      const char *const zeros = reinterpret_cast<const char *>(zero_row);
      const char *const q = p.io.q + (int64_t)p.seqs.q_begin(s) * p.io.q_stride + (int64_t)h * group * (D * 2);
#pragma unroll 4
      for (int r = threadIdx.x / kLanes; r < kTileRows; r += 256 / kLanes) {
        const int i = div_by(row0 + r, p.io.group), g = row0 + r - i * group;
        const char *src = row0 + r < rows ? q + i * p.io.q_stride + g * (D * 2) : zeros;
        cp_async16(smem_addr(q_smem) + (r >> 7) * Shape::kOperand + (c >> 3) * (kTileKeys * 128) + (r & 127) * 128 +
                       (((c & 7) ^ (r & 7)) << 4),
                   src + c * 16);
      }
      mbar_arrive_after_copies(&bars.q_full);
    }
    const int t = warp >> 2;
    const int in_block = (int)threadIdx.x, row = row0 + in_block;
    const int tile_first = row0 + t * 128;
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) * 32 << 16);
    const uint32_t s_at = lane_base + t * 128, o_at = lane_base + 256 + t * 128;
    const int token = div_by(row, p.io.group);
    const RowMask mask = row_mask(kv, nq, token, p.seqs.causal, p.seqs.window, p.seqs.sinks);
    int last = tile_first + 127;
    if (last >= rows) last = rows - 1;
    const int full_hi = row_mask(kv, nq, div_by(tile_first, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks).hi;
    const int full_lo = row_mask(kv, nq, div_by(last < 0 ? 0 : last, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks).lo;
    const float scale = p.io.scale_log2;
    float base = -INFINITY, l = 0.f;
    bool ok = true;
    const int my_n = t < tiles ? n : 0;
    for (int it = 0; it < my_n; ++it) {
      ok = tile_wait_warp(&bars, &bars.s_full[t], it & 1, status);
      if (!ok) break;
      tmem_fence_after();
      uint32_t x[4][32], w[2][16];
      tmem_load32(x[0], s_at);
      tmem_load32(x[1], s_at + 32);
      tmem_wait_loads(x[0]);
      tmem_wait_loads(x[1]);
      tmem_load32(x[2], s_at + 64);
      tmem_load32(x[3], s_at + 96);
      const int start = keys.tile_start(j0 + it, kTileKeys);
      const bool whole = start + kTileKeys <= full_hi && (start >= full_lo || start + kTileKeys <= p.seqs.sinks);
      auto largest = [&](int c) {
        float a = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
        float b = fmaxf(__uint_as_float(x[c][16]), __uint_as_float(x[c][17]));
#pragma unroll
        for (int i = 2; i < 16; i += 2) {
          a = max3(a, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
          b = max3(b, __uint_as_float(x[c][16 + i]), __uint_as_float(x[c][17 + i]));
        }
        return fmaxf(a, b);
      };
      // 2^(x scale - base) in place of the scores, and rounded
      auto weigh = [&](int c) {
        const float shift = base == -INFINITY ? 0.f : base;
        const uint64_t scale2 = pair(__float_as_uint(scale), __float_as_uint(scale));
        const uint64_t shift2 = pair(__float_as_uint(-shift), __float_as_uint(-shift));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = unpair(fma_pair(pair(x[c][2 * i], x[c][2 * i + 1]), scale2, shift2));
          const float a = exp2_approx(y.x), b = exp2_approx(y.y);
          w[c & 1][i] = pack2<T>(a, b);
          x[c][2 * i] = __float_as_uint(a);
          x[c][2 * i + 1] = __float_as_uint(b);
        }
      };
      // A new maximum: the sum and the output so far shrink by 2^(old - new).
      auto raise = [&](bool rise, float top) {
        const float next = rise ? top : base;
        const float fall = rise ? exp2_approx(base - next) : 1.f;
        base = next;
        l *= fall;
        if (it == 0) return;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_load32(o, o_at + c * 32);
          tmem_wait_loads(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fall);
          tmem_store32(o_at + c * 32, o);
        }
      };
      // With a maximum from before and nothing to mask, the first half's weights
      // are worked out for that maximum while the second half's scores arrive and
      // this tile's maximum is found: mostly the old one stands, and they do.
      const bool ahead = whole && __all_sync(0xffffffffu, base != -INFINITY);
      float top = 0.f;
      if (ahead) {
        top = fmaxf(largest(0), largest(1));
      } else {
        tmem_wait_loads(x[2]);
        tmem_wait_loads(x[3]);
        if (!whole) {
          const int lo = mask.lo - start, hi = mask.hi - start, sinks = mask.sinks - start;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int j = c * 32 + i;
              if (!(j < hi && (j >= lo || j < sinks))) x[c][i] = 0xff800000u;
            }
        }
        top = fmaxf(fmaxf(largest(0), largest(1)), fmaxf(largest(2), largest(3))) * scale;
        const bool rise = top > base + kRescaleAt || (base == -INFINITY && top != -INFINITY);
        if (__any_sync(0xffffffffu, rise)) raise(rise, top);
      }
      weigh(0);
      weigh(1);
      if (ahead) {
        tmem_wait_loads(x[2]);
        tmem_wait_loads(x[3]);
        top = fmaxf(top, fmaxf(largest(2), largest(3))) * scale;
        const bool rise = top > base + kRescaleAt;
        if (__any_sync(0xffffffffu, rise)) {
          raise(rise, top);
          tmem_load32(x[0], s_at);
          tmem_load32(x[1], s_at + 32);
          tmem_wait_loads(x[0]);
          tmem_wait_loads(x[1]);
          weigh(0);
          weigh(1);
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half == 1) {
          weigh(2);
          weigh(3);
        }
        tmem_store16(s_at + half * 32, w[0]);
        tmem_store16(s_at + half * 32 + 16, w[1]);
        tmem_wait_stores();
        tmem_fence_before();
        mbar_arrive(&bars.p_full[t][half]);
      }
      // the sum, beside the products
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[c] = add_pair(sum[c], pair(x[c][2 * i], x[c][2 * i + 1]));
      const float2 all = unpair(add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3])));
      l += all.x + all.y;
    }
    if (ok && my_n > 0) ok = tile_wait_warp(&bars, &bars.o_full[t], 0, status);
    tmem_fence_after();
    if (ok) {
      const int64_t slot_row = ((int64_t)item * splits + split) * kTileRows + in_block;
      const int head = h * group + row - token * group;
      const int64_t out_token = p.seqs.q_begin(s) + token;
      if (row < rows) {
        if (!p.direct) {
          *reinterpret_cast<float2 *>(p.space.ml + slot_row * 2) = make_float2(base, l);
        } else if (p.io.lse != nullptr) {
          p.io.lse[out_token * p.io.q_heads + head] = row_lse(base, l);
        }
      }
      const float inv = row_scale(l);
      char *dst = p.io.out + out_token * p.io.out_stride + (int64_t)head * (D * 2);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (my_n > 0) {
          tmem_load32(o, o_at + c * 32);
          tmem_wait_loads(o);
        }
        if (row >= rows) continue;
        if (p.direct) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = l == 0.f ? 0u : pack2<T>(__uint_as_float(o[v * 8 + 2 * e]) * inv, __uint_as_float(o[v * 8 + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4 *>(dst + c * 64 + v * 16) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else if (my_n > 0) {
          float *to = p.space.o + slot_row * D + c * 32;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *reinterpret_cast<uint4 *>(to + v * 4) = make_uint4(o[v * 4], o[v * 4 + 1], o[v * 4 + 2], o[v * 4 + 3]);
        }
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- loads
    // A lane looks up one key; its warp brings in those 32 keys.  Without a box it
    // leaves the address in shared memory and copies one 16-byte chunk of several
    // keys.  Keys that no query of the sequence sees are copied from zeros.
    shrink_registers<kOtherRegisters>();
    const KeyRange there = key_range<kTileKeys>(kv, nq, 0, nq, p.seqs.causal, p.seqs.window, p.seqs.sinks);
    const int lw = warp - 8;
    constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
    const int c = lane % kLanes;
    const int64_t k_at = p.io.k_off + (int64_t)h * D * 2, v_at = p.io.v_off + (int64_t)h * D * 2;
    const int32_t *pages = p.seqs.pages(s);
    const char *const zeros = reinterpret_cast<const char *>(zero_row);
    ulonglong2 *mine = addresses + lw * 32;
    const ulonglong2 *theirs = mine + lane / kLanes;
    uint32_t to[8 / kRowsAtOnce];  // this lane's places repeat every 8 keys
#pragma unroll
    for (int e = 0; e < 8 / kRowsAtOnce; ++e) {
      const int r = e * kRowsAtOnce + lane / kLanes;
      to[e] = (c >> 3) * (kTileKeys * 128) + (lw * 32 + r) * 128 + (((c & 7) ^ (r & 7)) << 4);
    }
    int key = 0, page = -1;
    auto look_up = [&](int j) {  // one tile ahead of its copies
      key = keys.tile_start(j, kTileKeys) + lw * 32 + lane;
      if (!there.any_sees(key)) key = -1;
      page = key >= 0 ? pages[div_by(key, p.pools.page_size)] : -1;
    };
    auto copy = [&](const char *operand, bool values) {
      const uint32_t base = smem_addr(operand);
#pragma unroll
      for (int g = 0; g < 32 / kRowsAtOnce; ++g) {
        const unsigned long long src = values ? theirs[g * kRowsAtOnce].y : theirs[g * kRowsAtOnce].x;
        cp_async16(base + to[g % (8 / kRowsAtOnce)] + g / (8 / kRowsAtOnce) * 1024,
                   reinterpret_cast<const char *>(src) + c * 16);
      }
    };
    // this lane's box of the warp's: block of 64 elements, first key
    const int boxes = p.box_rows ? 32 / p.box_rows * (D / 64) : 0;
    const int box_block = lane % (D / 64), box_key = lane / (D / 64) * p.box_rows;
    bool ok = true;
    if (n > 0) look_up(j0);
    for (int it = 0; it < n && ok; ++it) {
      int owner = 0, pool_row = 0;
      const char *at = nullptr;
      if (key >= 0) {
        const int in_page = key - div_by(key, p.pools.page_size) * (int)p.pools.page_size.d;
        at = page_address(p.pools, page);
        if (at == nullptr) {
          raise_status(status, CPKV_STATUS_PAGE_OOB);
        } else {
          at += (int64_t)in_page * p.pools.row_bytes;
          const int local = div_by(page, p.pools.cp);
          owner = page - local * (int)p.pools.cp.d;
          pool_row = local * (int)p.pools.page_size.d + in_page;
        }
      }
      const bool by_box = boxes > 0 && __all_sync(0xffffffffu, at != nullptr);
      if (by_box) {
        owner = __shfl_sync(0xffffffffu, owner, box_key);
        pool_row = __shfl_sync(0xffffffffu, pool_row, box_key);
      } else {
        __syncwarp();
        mine[lane] = make_ulonglong2((unsigned long long)(at == nullptr ? zeros : at + k_at),
                                     (unsigned long long)(at == nullptr ? zeros : at + v_at));
        __syncwarp();
      }
      if (it + 1 < n) look_up(j0 + it + 1);
      const int stage = it % kStages;
      const uint32_t freed = (it / kStages - 1) & 1;
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {  // keys, then values
        uint64_t *full = which ? &bars.v_full[stage] : &bars.k_full[stage];
        if (it >= kStages) ok = tile_wait_warp(&bars, which ? &bars.v_empty[stage] : &bars.k_empty[stage], freed, status);
        if (!ok) break;
        char *operand = (which ? v_smem : k_smem) + stage * Shape::kOperand;
        if (by_box) {
          if (lane < boxes) {
            mbar_arrive_expect_tx(full, (uint32_t)p.box_rows * 128);
            box_load(operand + box_block * (kTileKeys * 128) + (lw * 32 + box_key) * 128, &p.maps[owner],
                     (int)((which ? v_at : k_at) >> 1) + box_block * 64, pool_row, full);
          } else {
            mbar_arrive(full);
          }
        } else {
          copy(operand, which);
          mbar_arrive_after_copies(full);
        }
      }
    }
    cp_async_wait_all();
  } else {
    // ---------------------------------------------------------------- products
    // The copies are ordinary writes to shared memory: the fence of the thread
    // that issues the products (after the wait that orders them before it) lets
    // the tensor core see them.
    shrink_registers<kOtherRegisters>();
    if (__shfl_sync(0xffffffffu, warp, 0) == 12 && n > 0) {
      constexpr uint32_t desc_s = product_desc(kBf16, 128, kTileKeys, false), desc_o = product_desc(kBf16, 128, D, true);
      const uint32_t q_low = operand_low(smem_addr(q_smem), 16), k_low = operand_low(smem_addr(k_smem), 16);
      const uint32_t v_low = operand_low(smem_addr(v_smem), kTileKeys * 128);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int count = __shfl_sync(0xffffffffu, n, 0), row_tiles = __shfl_sync(0xffffffffu, tiles, 0);
      auto scores = [&](int t, int stage) {
        const uint32_t a = q_low + t * (Shape::kOperand >> 4), b = k_low + stage * (Shape::kOperand >> 4);
        const uint32_t d = tm + t * 128;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k >> 2) * (kTileKeys * 128) + (k & 3) * 32) >> 4;
            mma_ss(d, a + at, b + at, desc_s, k > 0);
          }
          mma_commit(&bars.s_full[t]);
        }
        __syncwarp();
      };
      auto values = [&](int t, int stage, int half, uint32_t add) {
        const uint32_t b = v_low + stage * (Shape::kOperand >> 4) + half * (64 * 128 >> 4);
        const uint32_t d = tm + 256 + t * 128, a = tm + t * 128 + half * 32;
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mma_ts(d, a + e * 8, b + e * (16 * 128 >> 4), desc_o, e > 0 ? 1 : add);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t *bar) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      bool ok = tile_wait_warp(&bars, &bars.q_full, 0, status);
      if (ok) ok = tile_wait_warp(&bars, &bars.k_full[0], 0, status);
      if (ok) {
        fence_proxy_async_smem();
        for (int t = 0; t < row_tiles; ++t) scores(t, 0);
        commit(&bars.k_empty[0]);
      }
      int stage = 0, phase = 0;
      for (int it = 0; it < count && ok; ++it) {
        const int next = stage + 1 == kStages ? 0 : stage + 1, next_phase = next == 0 ? phase ^ 1 : phase;
        ok = tile_wait_warp(&bars, &bars.v_full[stage], phase, status);
        if (it + 1 < count && ok) ok = tile_wait_warp(&bars, &bars.k_full[next], next_phase, status);
        fence_proxy_async_smem();
        for (int t = 0; t < row_tiles && ok; ++t) {
          for (int half = 0; half < 2 && ok; ++half) {
            ok = tile_wait_warp(&bars, &bars.p_full[t][half], it & 1, status);
            if (!ok) break;
            tmem_fence_after();
            values(t, stage, half, half > 0 || it > 0);
          }
          if (!ok) break;
          if (t == row_tiles - 1) commit(&bars.v_empty[stage]);
          if (it + 1 < count) scores(t, next);
        }
        if (ok && it + 1 < count) commit(&bars.k_empty[next]);
        stage = next;
        phase = next_phase;
      }
      commit(&bars.o_full[0]);
      commit(&bars.o_full[1]);
      if (!ok) {  // products in flight end before tensor memory is freed
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&bars.o_full[0], 0) && global_timer_ns() - t0 < kTileWaitNs) {
        }
      }
    }
    __syncwarp();
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 12) tmem_free(tmem, 512);
}

}  // namespace cpkv
