// Attention of many query rows on the tensor core: an item is 256 packed rows of
// one sequence and key/value head, which go once over the keys they see (or over one
// part of them), 128 at a time, with the running maximum and sum of each row's softmax.
//
// Two products per 128 keys, 4 * 256 * 128 * D operations on 2 * 128 * D values:
// the tensor core bounds it at D = 128, the exponentials (one per query and key)
// at D = 64.  The 256 rows are two tiles of 128 so that one tile's softmax runs
// while the tensor core multiplies for the other:
//   warps 0..3, 4..7   the softmax of tile 0, 1: a thread owns a row.  Scores come
//                      from tensor memory; weights go back over them, rounded to
//                      the element type (summed after that, beside the products).
//   warps 8..11        keys and values of the pages to shared memory, 32 keys each:
//                      as TMA boxes where a page holds 16 rows or more and all 32
//                      keys are there, else by cp.async with an address per key, so
//                      pages may have any size and stand in any order.
//   warp 12            issues the products: scores (queries, keys in shared memory),
//                      then values (weights in tensor memory), tile by tile.
//   warp 13            finds the next item while this one runs: the grid has a block
//                      for every item, and a running block claims blocks that have not
//                      started (cluster launch control), a request's later rows, which
//                      see more keys, before its earlier ones, so that no SM waits for
//                      another.  Requests go by number, whatever their lengths.
//   warps 14, 15       the next item's queries: two blocks of 128 rows, of which an item
//                      of at most 128 rows takes one, the items in turn.
// Over quantised rows (of few row tiles: many are read back first, attend_unpack.cuh) eight
// warps load, from the ninth on, and the others follow; they bring a key's e4m3 elements, times
// its scale, into shared memory in the element type, and the softmax holds half a row of scores
// at a time, for the registers that they take.
// Of an item with at most 128 rows the two tiles are the same rows over every other
// 128 keys (two streams), joined at the end.
// Tensor memory (512 columns): scores of the tiles at 0 and 128, outputs at 256
// and 384.  A row's output is rescaled only when its maximum has risen by more
// than 2^8 since the last time: weights stay below 2^8 (times kLift's factor), and the
// sum and the output carry the same factor, which cancels at the end.
// Measured: 44600 tokens of 12 requests, 32 heads of 128 on 8, a window of 4096 and 64
// sinks behind prefixes of up to 16384, take 2.12 ms: 1.41 PFLOP/s on the visible keys,
// 74% of the measured bf16 rate of plain products (the tensor pipe is busy 60% of the
// cycles of a causal prefill of 2 x 4096, whose diagonals it multiplies in full).  One
// decode step of 256 requests on a prefix of 65536: 0.55 ms, 1.02 PFLOP/s.
// With the products issued by one lane of a diverged warp, or operands worked out by
// it, the same prefill took 2.65 ms, with copies by cp.async alone 4.0 ms.
// Quantised rows: 5 requests of 64 tokens on 8192 keys in 60 us (the tensor pipe is busy 37%
// of a cold one's 68): the conversion's instructions and the softmax's bound it together.
#pragma once

#include <cuda.h>

#include "attend.cuh"
#include "quantised.cuh"
#include "tcgen05.cuh"

namespace cpkv {

constexpr int kTileRows = 256;  // packed rows of a block
constexpr int kTileKeys = 128;
// Warps: 8 of the softmax, then those that load, then four that issue products, find items
// and load queries.  Quantised rows are converted on the way and take eight warps.
constexpr int load_warps(bool quantised) { return quantised ? 8 : 4; }
constexpr int tile_threads(bool quantised) { return 32 * (12 + load_warps(quantised)); }
// Registers a thread: 512 threads are launched with 128 each, 65536 in all; the
// softmax holds a row's 128 scores.  256 * 216 + 256 * 40 = 65536.
constexpr int kSoftmaxRegisters = 216, kOtherRegisters = 40;
// Over quantised rows 640 threads are launched with 96 each, 61440 in all, and the softmax
// holds half a row's scores: 256 * 152 + 256 * 64 + 128 * 48 = 61440.
constexpr int kSoftmaxRegistersQ = 152, kLoadRegistersQ = 64, kOtherRegistersQ = 48;
constexpr int kTurn = 2;  // passes (16 elements a lane) that a loading warp converts together
constexpr int kItemSlots = 4;   // items known at a time: of small ones, some are loaded while others are finished
constexpr int kClaimAhead = 12;  // key tiles before an item's last load at which the next item is claimed
constexpr int kTileMaps = 8;  // most pools that TMA maps travel for
constexpr float kRescaleAt = 8.f;
constexpr uint64_t kTileWaitNs = 2000000000ull;  // and, for each key tile of an item,
constexpr uint64_t kTileStepNs = 50000;          // of which one takes about 1.4 us
constexpr uint32_t kTileParkNs = 2000;
constexpr uint64_t kTileDrainNs = 50000000ull;  // for copies and products in flight after giving up: they take microseconds

// Rows of a tile pass's parts: 256 for each [item][split], an item being (row tile
// of the ragged sequences, key/value head), then those of the sequences of one
// query, [sequence][key/value head][row tile][split] of its rows.
struct TileSpace {
  float *ml;  // [row][2]
  float *o;   // [row][D]
  int splits, single_splits;
  int items;           // of the ragged sequences
  int single_tiles;    // row tiles of a sequence of one query
  int64_t single_row;  // where their rows begin
  FastDiv by_heads, by_splits, by_single_splits, by_single_tiles;
};

template <typename S>
struct TileParams {
  S seqs;
  PagedPools pools;
  AttendIo io;
  TileSpace space;
  int direct;           // one split, and the rows go straight to the output
  int wide_out;         // the output's rows start on 32 bytes
  int box_rows;         // rows of a TMA box (32 or 16); 0: no maps
  int cu_tiles[S::kArray + 1];  // row tiles before each ragged sequence
  uint64_t test_wait_ns;  // limit of the waits in the self-test of giving up
  CUtensorMap maps[kTileMaps];  // pool r as [rows][elements], boxes of box_rows x 64
};

// Finds the parts of a row of a tile pass.
template <typename S>
struct TileSource {
  S seqs;
  TileSpace space;
  int cu_tiles[S::kArray + 1];
};

// Rows of a part of a sequence of one query.
CPKV_DEV int single_rows(int group) { return group < kTileRows ? group : kTileRows; }

template <int D, bool kQuantised>
struct TileShape {
  static constexpr int kOperand = kTileKeys * D * 2;  // keys (or values, or 128 queries) in shared memory
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kQ = 2 * kOperand;
  static constexpr int kRawTurns = 3;  // turns of quantised rows in a loading warp's ring
  static constexpr int kRaw = kQuantised ? load_warps(true) * kRawTurns * kTurn * 512 : 0;
  static constexpr int kSmem = 1024 + kQ + 2 * kStages * kOperand + kRaw;
};

// What the warps of a block are told of an item.
struct TileItem {
  int more;  // 0: no item, the block ends
  int h, row0, rows, group_tiles, kv, nq, n, j0, streams;
  int64_t q_begin, slot;  // first query token; first row of its parts
  const int32_t *pages;
  KeyRange keys;   // what the item's rows see
  KeyRange there;  // what the sequence's rows see: present in the pools
};

struct TileBars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], o_full[2], q_full[2], q_empty[2];
  uint64_t item_full[kItemSlots], item_empty[kItemSlots], wanted, claimed, drain, stream_done, stream_free;
  uint4 claim;
  uint32_t tmem;
  int gave_up;
  int loaders;        // warps that may issue copies
  uint64_t deadline;  // of the waits; moves on with the items
  uint32_t issued[4];  // keys and values of tiles, in turn, that a loading warp has issued
};

constexpr int item_readers(bool quantised) { return 11 + load_warps(quantised); }  // warps that read an item: softmax, loads, products, queries

__device__ const uint4 zero_row[16] = {};  // a key or value vector of zeros

// Bounded wait of a thread: whether the phase came.  When it did not before the
// deadline, or another wait of the block ran out, the block gives up: loads and claims
// end at once (kStops), the other roles run through what they have begun on whatever is
// there once no copy is issued any more (a stage that they hand back unseen is not filled
// again), what is in flight is waited for, and the status word says that the results are
// undefined.
// The usual way through is one instruction and one branch: the products' warp does
// nine waits per 128 keys, and its own pace is close to the tensor core's.  A branch on
// the result in its loop cost 1.6% of a prefill, a deadline that a loading warp moves on
// every 64 tiles 2.7%: the warp that finds the items keeps it.
template <bool kTest, bool kStops>
CPKV_DEV bool tile_wait(TileBars *b, uint64_t *bar, uint32_t parity, int32_t *status) {
  constexpr uint32_t kPark = kTest ? 0 : kTileParkNs;
  if (mbar_try_wait_for(bar, parity, kPark)) return true;
  while (!mbar_try_wait_for(bar, parity, kPark)) {
    if (!*(volatile int *)&b->gave_up) {
      if (global_timer_ns() <= *(volatile uint64_t *)&b->deadline) continue;
      *(volatile int *)&b->gave_up = 1;
      raise_status(status, CPKV_STATUS_TIMEOUT);
    }
    if (kStops) return false;
    const uint64_t t0 = global_timer_ns();
    while (*(volatile int *)&b->loaders > 0 && global_timer_ns() - t0 < kTileDrainNs) {
    }
    return false;
  }
  return true;
}

// Waits for a phase that something in flight completes, no longer than kTileDrainNs from t0.
CPKV_DEV void tile_drain(uint64_t *bar, uint32_t parity, uint64_t t0) {
  while (!mbar_try_wait(bar, parity & 1) && global_timer_ns() - t0 < kTileDrainNs) {
  }
}

// The lowest n bits, n clamped to 0..32.
CPKV_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

// The item of a block index: the ragged sequences' last row tiles first, which see
// the most keys, then the sequences of one query.
template <typename S>
CPKV_DEV void find_item(const TileParams<S> &p, int block, TileItem *r) {
  const int heads = p.io.kv_heads, group = p.io.group.d, many = p.space.items * p.space.splits;
  int s, rt, splits, split;
  if (block < many) {
    splits = p.space.splits;
    const int cut = div_by(block, p.space.by_splits), index = p.space.items - 1 - cut;
    const int tile = div_by(index, p.space.by_heads);
    split = block - cut * splits;
    s = upper_index(p.cu_tiles, p.seqs.ragged(), tile);
    rt = tile - p.cu_tiles[s];
    r->h = index - tile * heads;
    r->slot = ((int64_t)index * splits + split) * kTileRows;
  } else {
    splits = p.space.single_splits;
    const int rest = block - many, index = div_by(rest, p.space.by_single_splits);
    const int y = div_by(index, p.space.by_single_tiles), of = div_by(y, p.space.by_heads);
    split = rest - index * splits;
    s = p.seqs.ragged() + of;
    rt = index - y * p.space.single_tiles;
    r->h = y - of * heads;
    r->slot = p.space.single_row + (int64_t)rest * single_rows(group);
  }
  r->nq = p.seqs.q_count(s);
  r->kv = p.seqs.kv_len(s);
  r->rows = r->nq * group;
  r->row0 = rt * kTileRows;
  r->q_begin = p.seqs.q_begin(s);
  r->pages = p.seqs.pages(s);
  const int end = r->row0 + kTileRows < r->rows ? r->row0 + kTileRows : r->rows;
  r->keys = key_range<kTileKeys>(r->kv, r->nq, div_by(r->row0, p.io.group), div_by(end - 1, p.io.group) + 1, p.seqs.causal,
                                 p.seqs.window, p.seqs.sinks);
  r->there = key_range<kTileKeys>(r->kv, r->nq, 0, r->nq, p.seqs.causal, p.seqs.window, p.seqs.sinks);
  r->j0 = 0;
  r->n = r->keys.n_tiles;
  if (splits > 1) {  // fewer than 2^24 key tiles, at most some hundred parts
    r->j0 = (int)((uint32_t)r->keys.n_tiles * (uint32_t)split / (uint32_t)splits);
    r->n = (int)((uint32_t)r->keys.n_tiles * (uint32_t)(split + 1) / (uint32_t)splits) - r->j0;
  }
  r->group_tiles = end - r->row0 > 128 ? 2 : 1;
  r->streams = r->group_tiles == 1 ? 2 : 1;
  r->more = 1;
  if (split == 0 && r->h == 0 && rt == 0 && p.seqs.kv_len_bad(s)) raise_status(p.seqs.status, CPKV_STATUS_OUT_CAPACITY);
}

// x.y + sum and o + w v, two elements each.
template <typename T>
CPKV_DEV float add_product(uint32_t x, uint32_t y, float sum) {
  const float2 a = unpack2<T>(x), b = unpack2<T>(y);
  return fmaf(a.x, b.x, fmaf(a.y, b.y, sum));
}
template <typename T>
CPKV_DEV void add_scaled(float *o, float w, uint32_t v) {
  const float2 b = unpack2<T>(v);
  o[0] = fmaf(w, b.x, o[0]);
  o[1] = fmaf(w, b.y, o[1]);
}

// A row of an item whose output holds a NaN, by the thread that wrote it.  A product
// adds weight 0 times the value for keys of a tile that the row does not see, so where
// one of those values is infinite or a NaN the output is worked out again over the keys
// that it does see, with the maximum and sum that the row has (which no other key
// enters): to `out` (16-bit results) or `part` (a part's values).  For NaNs only: to look
// at the values beforehand costs more (traced prefill 2.27 ms where it is 2.13).
// Latency bounds it: an item whose 256 rows all need it takes 3.1 us a key (19 a key at a
// time; four in flight together), so the block's waits are given more time meanwhile.
// Eight rows at a time over a warp's lanes took 2.1 us a key, but the kernel that called
// it, without calling it, took 8% longer.
constexpr int kMendKeys = 4;  // at a time

// A key's vectors in memory, 8 elements at a time.
template <typename T, bool kQuantised>
struct RowVector {
  const char *at;  // zero_row for none
  float scale;
  CPKV_DEV uint4 operator[](int c) const {
    if constexpr (kQuantised) return read_back8<T>(reinterpret_cast<const uint2 *>(at)[c], scale);
    return reinterpret_cast<const uint4 *>(at)[c];
  }
};

template <typename T, int D, typename S, bool kQuantised>
__device__ __noinline__ void mend_row(const TileParams<S> &p, const TileItem &item, uint64_t *deadline, int token, int head, float base, float l,
                                      char *out, float *part) {
  const RowMask mask = row_mask(item.kv, item.nq, token, p.seqs.causal, p.seqs.window, p.seqs.sinks);
  using Vector = RowVector<T, kQuantised>;
  constexpr int kBytes = D * (kQuantised ? 1 : 2);  // of a vector
  const int64_t k_at = p.io.k_off + (int64_t)item.h * kBytes, v_at = p.io.v_off + (int64_t)item.h * kBytes;
  auto row_of = [&](int key) -> const char * {
    const int page = div_by(key, p.pools.page_size);
    const char *const at = page_address(p.pools, item.pages[page]);
    return at == nullptr ? nullptr : at + (int64_t)(key - page * (int)p.pools.page_size.d) * p.pools.row_bytes;
  };
  auto scale_of = [&](const char *row, int64_t off) {
    if constexpr (kQuantised) return *reinterpret_cast<const float *>(row + off + (int64_t)item.h * 4);
    return 1.f;
  };
  uint4 marks = make_uint4(0, 0, 0, 0);
  for (int j = item.j0; j < item.j0 + item.n; ++j) {
    const int start = item.keys.tile_start(j, kTileKeys);
    if (start + kTileKeys <= mask.hi && (start >= mask.lo || start + kTileKeys <= mask.sinks)) continue;
    for (int key = start; key < start + kTileKeys; ++key) {
      if (mask.sees(key) || !item.there.any_sees(key)) continue;
      const char *const at = row_of(key);
      if (at == nullptr) continue;
      const Vector v = {at + v_at, scale_of(at, p.io.vs_off)};
#pragma unroll
      for (int c = 0; c < D / 8; ++c) marks = mark_infinite<T>(v[c], marks);
    }
  }
  if ((marks.x | marks.y | marks.z | marks.w) == 0) return;  // its NaNs are its own

  const char *const q = p.io.q + (item.q_begin + token) * p.io.q_stride + (int64_t)head * (D * 2);
  const float shift = base == -INFINITY ? 0.f : base, inv = row_scale(l);
#pragma unroll 1
  for (int half = 0; half < D / 64; ++half) {
    float o[64] = {};
    for (int j = item.j0; j < item.j0 + item.n; ++j) {
      const int start = item.keys.tile_start(j, kTileKeys);
      atomicMax(reinterpret_cast<unsigned long long *>(deadline), (unsigned long long)(global_timer_ns() + kTileWaitNs));
#pragma unroll 1
      for (int first = start; first < start + kTileKeys; first += kMendKeys) {
        Vector k[kMendKeys], v[kMendKeys];  // vectors of zeros for keys that the row does not see
        float w[kMendKeys] = {};
        uint32_t seen = 0;
#pragma unroll
        for (int i = 0; i < kMendKeys; ++i) {
          const char *const at = mask.sees(first + i) ? row_of(first + i) : nullptr;
          const char *const none = reinterpret_cast<const char *>(zero_row);
          k[i] = at != nullptr ? Vector{at + k_at, scale_of(at, p.io.ks_off)} : Vector{none, 0.f};
          v[i] = at != nullptr ? Vector{at + v_at + half * (kBytes / (D / 64)), scale_of(at, p.io.vs_off)} : Vector{none, 0.f};
          seen |= at != nullptr ? 1u << i : 0u;
        }
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
          const uint4 a = reinterpret_cast<const uint4 *>(q)[c];
#pragma unroll
          for (int i = 0; i < kMendKeys; ++i) {
            const uint4 b = k[i][c];
            w[i] = add_product<T>(a.x, b.x, add_product<T>(a.y, b.y, add_product<T>(a.z, b.z, add_product<T>(a.w, b.w, w[i]))));
          }
        }
#pragma unroll
        for (int i = 0; i < kMendKeys; ++i) w[i] = seen >> i & 1 ? exp2_approx(fmaf(w[i], p.io.scale_log2, -shift)) : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
          for (int i = 0; i < kMendKeys; ++i) {
            const uint4 b = v[i][c];
            add_scaled<T>(o + 8 * c, w[i], b.x);
            add_scaled<T>(o + 8 * c + 2, w[i], b.y);
            add_scaled<T>(o + 8 * c + 4, w[i], b.z);
            add_scaled<T>(o + 8 * c + 6, w[i], b.w);
          }
      }
    }
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (part != nullptr) {
        reinterpret_cast<float2 *>(part + half * 64)[c] = make_float2(o[2 * c], o[2 * c + 1]);
      } else {
        reinterpret_cast<uint32_t *>(out + half * 128)[c] = pack2<T>(o[2 * c] * inv, o[2 * c + 1] * inv);
      }
    }
  }
}

template <typename T, int D, typename S, bool kTest, bool kQuantised>
__global__ void __launch_bounds__(tile_threads(kQuantised), 1) attend_tile_kernel(const __grid_constant__ TileParams<S> p) {
  using Shape = TileShape<D, kQuantised>;
  constexpr int kStages = Shape::kStages;
  constexpr int kLoadWarps = load_warps(kQuantised), kProducts = 8 + kLoadWarps;  // the warp that issues products
  constexpr int kOthers = kQuantised ? kOtherRegistersQ : kOtherRegisters;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ char raw_smem[];
  __shared__ TileBars bars;
  __shared__ TileItem items[kItemSlots];
  __shared__ float2 stream_ml[128];            // maximum and sum of the second stream's rows
  __shared__ ulonglong2 addresses[kQuantised ? 1 : kTileKeys];  // of the keys being copied: key, value
  char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  char *q_smem = smem, *k_smem = smem + Shape::kQ, *v_smem = k_smem + kStages * Shape::kOperand;
  [[maybe_unused]] char *const pieces = v_smem + kStages * Shape::kOperand;  // the loading warps' rings of quantised rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t *status = p.seqs.status;
  release_dependents();  // later passes of the call; the joining kernel waits for this one

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.k_full[i], 32 * kLoadWarps);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 32 * kLoadWarps);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.o_full[t], 1);
      mbar_init(&bars.p_full[t], 128);
      mbar_init(&bars.q_full[t], 64);
      mbar_init(&bars.q_empty[t], 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(&bars.item_full[i], 1);
      mbar_init(&bars.item_empty[i], item_readers(kQuantised));
    }
    mbar_init(&bars.wanted, 1);
    mbar_init(&bars.claimed, 1);
    mbar_init(&bars.drain, 1);
    mbar_init(&bars.stream_done, 128);
    mbar_init(&bars.stream_free, 128);
    bars.gave_up = 0;
    bars.loaders = kLoadWarps;
    bars.deadline = ~uint64_t(0);  // until the first item is known
    fence_barrier_init();
  }
  if (warp == kProducts) tmem_alloc(&bars.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = bars.tmem;
  auto wait = [&](uint64_t *bar, uint32_t parity) { (void)tile_wait<kTest, false>(&bars, bar, parity & 1, status); };
  auto wait_or_stop = [&](uint64_t *bar, uint32_t parity) { return tile_wait<kTest, true>(&bars, bar, parity & 1, status); };
  auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  // Item number k of this block: whether there is one.  The warp reads it and hands
  // its place back.
  auto item_there = [&](int k) {
    wait_or_stop(&bars.item_full[k % kItemSlots], k / kItemSlots);
    return all(items[k % kItemSlots].more && !*(volatile int *)&bars.gave_up);
  };
  auto item_read = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.item_empty[k % kItemSlots]);
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    grow_registers<kQuantised ? kSoftmaxRegistersQ : kSoftmaxRegisters>();
    const int t = warp >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) * 32 << 16);
    const uint32_t s_at = lane_base + t * 128, o_at = lane_base + 256 + t * 128;
    const float scale = p.io.scale_log2;
    uint32_t seen = 0, done0 = 0, done1 = 0, pairs = 0;  // score tiles, outputs of the tiles, items of two streams
    for (int k = 0; item_there(k); ++k) {
      const TileItem &item = items[k % kItemSlots];  // kept until its results are written
      const int step = item.streams;
      const int my_n = step == 2 ? (item.n + 1 - t) / 2 : t < item.group_tiles ? item.n : 0;
      const int j0 = step == 2 ? item.j0 + t : item.j0;
      const int first = item.row0 + (step == 2 ? 0 : t * 128);
      const int n_sink = item.keys.n_sink, first_tile = item.keys.first_tile - n_sink;
      int whole_lo, whole_hi;  // keys that every row of the tile sees
      {
        const int last = first + 127 < item.rows ? first + 127 : item.rows - 1;
        whole_hi = row_mask(item.kv, item.nq, div_by(first, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks).hi;
        whole_lo = row_mask(item.kv, item.nq, div_by(last, p.io.group), p.seqs.causal, p.seqs.window, p.seqs.sinks).lo;
      }
      float base = -INFINITY, l = 0.f;
      for (int it = 0; it < my_n; ++it) {
        wait(&bars.s_full[t], seen);
        __syncwarp();
        tmem_fence_after();
        constexpr int kChunks = kQuantised ? 2 : 4;  // 32 columns each that are held at a time
        uint32_t x[kChunks][32];
        const int j = j0 + it * step, start = (j < n_sink ? j : first_tile + j) * kTileKeys;
        const bool partly = !(start + kTileKeys <= whole_hi && (start >= whole_lo || start + kTileKeys <= p.seqs.sinks));
        auto scores_of = [&](int from) {  // of columns from 32 * from on; -infinity where the row does not see the key
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_load32(x[c], s_at + (from + c) * 32);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tmem_wait_loads(x[c]);
          if (partly) {
            const RowMask mask = row_mask(item.kv, item.nq, div_by(first + (int)(threadIdx.x & 127), p.io.group), p.seqs.causal,
                                          p.seqs.window, p.seqs.sinks);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int at = start + (from + c) * 32;
              const uint32_t sees = low_bits(mask.hi - at) & (~low_bits(mask.lo - at) | low_bits(mask.sinks - at));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(sees & (1u << i))) x[c][i] = 0xff800000u;
            }
          }
        };
        float best[4];
        auto best_of = [&](int from) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            best[from + c] = fmaxf(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]));
#pragma unroll
            for (int i = 2; i < 32; i += 2) best[from + c] = max3(best[from + c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
          }
        };
        scores_of(0);
        best_of(0);
        if constexpr (kQuantised) {  // the first half is looked at once more: its registers are the loading warps'
          scores_of(2);
          best_of(2);
        }
        const float top = fmaf(fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])), scale, -kLift<T, true>);
        const bool rise = top > base + kRescaleAt || (base == -INFINITY && top != -INFINITY);
        if (__any_sync(0xffffffffu, rise)) {  // the sum and the output so far shrink by 2^(old - new)
          const float next = rise ? top : base;
          const float fall = rise ? exp2_approx(base - next) : 1.f;
          base = next;
          l *= fall;
          if (it > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_load32(o, o_at + c * 32);
              tmem_wait_loads(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fall);
              tmem_store32(o_at + c * 32, o);
            }
          }
        }
        const float shift = base == -INFINITY ? 0.f : base;
        const uint64_t scale2 = pair(__float_as_uint(scale), __float_as_uint(scale));
        const uint64_t shift2 = pair(__float_as_uint(-shift), __float_as_uint(-shift));
        auto weights = [&](int at) {  // over the scores, 32 columns of them in 16
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = unpair(fma_pair(pair(x[c][2 * i], x[c][2 * i + 1]), scale2, shift2));
              const float a = exp2_approx(y.x), b = exp2_approx(y.y);
              w[i] = pack2<T>(a, b);
              x[c][2 * i] = __float_as_uint(a);
              x[c][2 * i + 1] = __float_as_uint(b);
            }
            tmem_store16(s_at + at + c * 16, w);
          }
        };
        auto add_up = [&] {
          uint64_t sum[kChunks] = {};
#pragma unroll
          for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) sum[c] = add_pair(sum[c], pair(x[c][2 * i], x[c][2 * i + 1]));
          if constexpr (kChunks == 4) {
            const float2 all = unpair(add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3])));
            l += all.x + all.y;
          } else {
            const float2 all = unpair(add_pair(sum[0], sum[1]));
            l += all.x + all.y;
          }
        };
        if constexpr (kQuantised) {
          weights(64);
          add_up();
          scores_of(0);
        }
        weights(0);
        tmem_wait_stores();
        tmem_fence_before();
        mbar_arrive(&bars.p_full[t]);
        add_up();  // beside the products
        ++seen;
      }
      // outputs of the item: of both tiles, so that either thread keeps count
      const bool has0 = item.n > 0, has1 = step == 2 ? item.n > 1 : has0 && item.group_tiles == 2;
      float mine = 1.f, other = 0.f;  // factors of the first and second stream's outputs
      if (step == 2) {
        if (t == 1) {
          stream_ml[threadIdx.x & 127] = make_float2(base, l);
          mbar_arrive(&bars.stream_done);
          done0 += has0;
          done1 += has1;
          wait(&bars.stream_free, pairs++);
          item_read(k);
          continue;
        }
        wait(&bars.stream_done, pairs++);
        const float2 ml = stream_ml[threadIdx.x & 127];
        const float top = fmaxf(base, ml.x), shift = top == -INFINITY ? 0.f : top;
        mine = exp2_approx(base - shift);
        other = exp2_approx(ml.x - shift);
        l = l * mine + ml.y * other;
        base = top;
        if (has1) wait(&bars.o_full[1], done1);
      }
      if (t == 0 ? has0 : has1) wait(&bars.o_full[t], t == 0 ? done0 : done1);
      done0 += has0;
      done1 += has1;
      __syncwarp();
      tmem_fence_after();
      const int row = first + (int)(threadIdx.x & 127), rows = item.rows, token = div_by(row, p.io.group);
      const int head = item.h * (int)p.io.group.d + row - token * (int)p.io.group.d;
      const int64_t out_token = item.q_begin + token;
      const int64_t slot_row = item.slot + threadIdx.x;
      if (!S::causal) item_read(k);
      uint64_t marks = 0;  // 0 until an output is infinite or a NaN
      if (row < rows) {
        if (!p.direct) {
          *reinterpret_cast<float2 *>(p.space.ml + slot_row * 2) = make_float2(base, l);
        } else if (p.io.lse != nullptr) {
          p.io.lse[out_token * p.io.q_heads + head] = row_lse(base, l);
        }
      }
      if (__any_sync(0xffffffffu, row < rows)) {
        const float inv = row_scale(l);
        char *dst = p.io.out + out_token * p.io.out_stride + (int64_t)head * (D * 2);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          if (my_n > 0) {
            tmem_load32(o, o_at + c * 32);
            tmem_wait_loads(o);
          }
          if (step == 2 && has1) {  // the second stream's rows are in the same lanes
            uint32_t o1[32];
            tmem_load32(o1, o_at + 128 + c * 32);
            tmem_wait_loads(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), other, __uint_as_float(o[i]) * mine));
          }
          if (row >= rows) continue;
          if constexpr (S::causal) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) marks = fma_pair(pair(o[i], o[i + 1]), 0, marks);
          }
          // 32 bytes a store where they are aligned: a warp's rows lie apart, and each
          // store of it takes as long as it touches lines
          if (p.direct) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                y[e] = l == 0.f ? 0u
                                : pack2<T>(__uint_as_float(o[v * 16 + 2 * e]) * inv, __uint_as_float(o[v * 16 + 2 * e + 1]) * inv);
              if (p.wide_out) {
                store32(dst + c * 64 + v * 32, y);
              } else {
                *reinterpret_cast<uint4 *>(dst + c * 64 + v * 32) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4 *>(dst + c * 64 + v * 32 + 16) = make_uint4(y[4], y[5], y[6], y[7]);
              }
            }
          } else if (my_n > 0) {
            float *to = p.space.o + slot_row * D + c * 32;
#pragma unroll
            for (int v = 0; v < 4; ++v) store32(to + v * 8, o + v * 8);
          }
        }
      }
      tmem_fence_before();
      if (step == 2) mbar_arrive(&bars.stream_free);
      if constexpr (S::causal) {
        const float2 m = unpair(marks);
        const bool bad = row < rows && item.nq > 1 && my_n > 0 && !(m.x == 0.f && m.y == 0.f);
        if (bad)
          mend_row<T, D, S, kQuantised>(p, item, &bars.deadline, token, head, base, l,
                                        p.io.out + out_token * p.io.out_stride + (int64_t)head * (D * 2),
                                        p.direct ? nullptr : p.space.o + slot_row * D);
        item_read(k);
      }
    }
  } else if (warp < kProducts) {
    // ---------------------------------------------------------------- keys and values
    if constexpr (kQuantised) {
      // A lane has one key of the warp's 16 and half its vector (lanes 0..15 the first half):
      // it looks the key up and brings 16 e4m3 elements at a time by cp.async to a place of its own,
      // from there, times their scale and in the element type, into the operand, and shares
      // nothing with the other lanes.  Through registers alone the same loads took half as long
      // again: with this much shared memory in use, the first-level cache that they pass through
      // holds too few of them.  The instructions of the conversion (about 45 for 16 elements)
      // set the pace, beside the softmax's: a prefill of 3.02 ms took 3.06 with addresses and
      // scales shuffled between lanes, and 3.67 with four warps of them (2.13 over plain rows).
      shrink_registers<kLoadRegistersQ>();
      const int lw = warp - 8;
      constexpr int kKeys = kTileKeys / kLoadWarps, kPasses = D / 32;                 // of an operand
      constexpr int kTurns = 2 * kPasses / kTurn, kAhead = Shape::kRawTurns - 1;      // of a tile; on their way
      static_assert(kKeys == 16 && kPasses % kTurn == 0 && kAhead <= kTurns, "lanes, passes and turns");
      const int half = lane >> 4;
      char *const ring = pieces + lw * (Shape::kRawTurns * kTurn * 512) + lane * 16;
      // this lane's row of an operand; 16-byte chunk c of it lies at c ^ (row % 8)
      const int row = lw * kKeys + lane % kKeys;
      const int to = half * (D == 128 ? kTileKeys * 128 : 0) + row * 128 + ((row & 7) << 4), flip = D == 128 ? 0 : half * 64;
      bool ok = true;
      uint32_t loaded = 0;         // key tiles
      int fill = 0, empty = 0;     // places in the ring of the next turn to issue and to convert
      for (int k = 0; ok && item_there(k); ++k) {
        const TileItem &item = items[k % kItemSlots];
        const int n = item.n, j0 = item.j0, n_sink = item.keys.n_sink, first_tile = item.keys.first_tile;
        const int lo = item.there.lo, hi = item.there.hi, sink_end = item.there.sink_end;
        const int32_t *const pages = item.pages;
        const int h = item.h;
        item_read(k);
        int key = 0, page = -1;
        auto look_up = [&](int j) {  // this lane's key of a tile, and its page
          key = (j < n_sink ? j : first_tile + j - n_sink) * kTileKeys + row;
          if (!(key < sink_end || (key >= lo && key < hi))) key = -1;
          page = key >= 0 ? pages[div_by(key, p.pools.page_size)] : -1;
        };
        // of this lane's key in the tile that is issued: its half vectors (zeros where there is none) and scales
        const char *from[2] = {nullptr, nullptr};
        int bytes = 0;
        float k_scale = 0.f, v_scale = 0.f;
        auto resolve = [&] {
          const char *at = nullptr;
          if (key >= 0) {
            at = page_address(p.pools, page);
            if (at == nullptr) {
              raise_status(status, CPKV_STATUS_PAGE_OOB);
            } else {
              at += (int64_t)(key - div_by(key, p.pools.page_size) * (int)p.pools.page_size.d) * p.pools.row_bytes;
            }
          }
          const char *const zeros = reinterpret_cast<const char *>(zero_row);
          bytes = at == nullptr ? 0 : 16;
          from[0] = at == nullptr ? zeros : at + p.io.k_off + (h * D + half * (D / 2));
          from[1] = at == nullptr ? zeros : at + p.io.v_off + (h * D + half * (D / 2));
          k_scale = at == nullptr ? 0.f : __ldg(reinterpret_cast<const float *>(at + p.io.ks_off) + h);
          v_scale = at == nullptr ? 0.f : __ldg(reinterpret_cast<const float *>(at + p.io.vs_off) + h);
        };
        auto issue = [&](int turn, bool there) {  // turn of the tile in hand
          if (there) {
            const uint32_t dst = smem_addr(ring + fill * (kTurn * 512));
#pragma unroll
            for (int e = 0; e < kTurn; ++e) {
              const int pass = turn * kTurn + e;
              cp_async16_or_zeros(dst + e * 512, from[pass / kPasses] + pass % kPasses * 16, bytes);
            }
            fill = fill + 1 == Shape::kRawTurns ? 0 : fill + 1;
          }
          cp_async_commit();
        };
        if (n > 0) {
          look_up(j0);
          resolve();
#pragma unroll
          for (int turn = 0; turn < kAhead; ++turn) issue(turn, true);
          if (n > 1) look_up(j0 + 1);
        }
        for (int it = 0; it < n; ++it) {
          const int stage = loaded % kStages;
          const bool reuse = loaded >= kStages, more = it + 1 < n;
          const uint32_t freed = (loaded / kStages - 1) & 1;
          ++loaded;
          const float ks = k_scale, vs = v_scale;
#pragma unroll
          for (int turn = 0; turn < kTurns; ++turn) {
            if (turn + kAhead == kTurns && more) {  // what is issued from here on is the next tile's
              resolve();
              if (it + 2 < n) look_up(j0 + it + 2);
            }
            const int which = turn * kTurn / kPasses;  // keys, then values
            if (turn * kTurn % kPasses == 0) {
              ok = all(!reuse || wait_or_stop(which ? &bars.v_empty[stage] : &bars.k_empty[stage], freed));
              if (!ok) break;
            }
            issue((turn + kAhead) % kTurns, turn + kAhead < kTurns || more);
            cp_async_wait<kAhead>();
            uint4 x[kTurn];
#pragma unroll
            for (int e = 0; e < kTurn; ++e) x[e] = *reinterpret_cast<const uint4 *>(ring + empty * (kTurn * 512) + e * 512);
            empty = empty + 1 == Shape::kRawTurns ? 0 : empty + 1;
            char *const operand = (which ? v_smem : k_smem) + stage * Shape::kOperand;
            const float s = which ? vs : ks;
#pragma unroll
            for (int e = 0; e < kTurn; ++e) {
              const int c = (turn * kTurn + e) % kPasses * 2;  // the first of this half's two chunks of 8 elements
              *reinterpret_cast<uint4 *>(operand + (to ^ (flip + c * 16))) = read_back8<T>(make_uint2(x[e].x, x[e].y), s);
              *reinterpret_cast<uint4 *>(operand + (to ^ (flip + c * 16 + 16))) = read_back8<T>(make_uint2(x[e].z, x[e].w), s);
            }
            if ((turn + 1) * kTurn % kPasses == 0) mbar_arrive(which ? &bars.v_full[stage] : &bars.k_full[stage]);
          }
          if (!ok) break;
          if (warp == 8 && lane == 0 && it == (n > kClaimAhead ? n - kClaimAhead : 0)) mbar_arrive(&bars.wanted);
        }
        if (warp == 8 && lane == 0 && n == 0) mbar_arrive(&bars.wanted);
      }
      cp_async_wait_all();
      if (lane == 0) atomicSub(&bars.loaders, 1);
    } else {
      // A lane looks up one key; its warp brings in those 32 keys.  Without a box it
      // leaves the address in shared memory and copies one 16-byte chunk of several
      // keys.  Keys that no query of the sequence sees are copied from zeros.
      shrink_registers<kOtherRegisters>();
      const int lw = warp - 8;
      constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
      const int c = lane % kLanes;
      const char *const zeros = reinterpret_cast<const char *>(zero_row);
      ulonglong2 *mine = addresses + lw * 32;
      const ulonglong2 *theirs = mine + lane / kLanes;
      uint32_t to[8 / kRowsAtOnce];  // this lane's places repeat every 8 keys
#pragma unroll
      for (int e = 0; e < 8 / kRowsAtOnce; ++e) {
        const int r = e * kRowsAtOnce + lane / kLanes;
        to[e] = (c >> 3) * (kTileKeys * 128) + (lw * 32 + r) * 128 + (((c & 7) ^ (r & 7)) << 4);
      }
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
      uint32_t operands = 0;
      for (int k = 0; ok && item_there(k); ++k) {
        const TileItem &item = items[k % kItemSlots];
        const int n = item.n, j0 = item.j0, n_sink = item.keys.n_sink, first_tile = item.keys.first_tile;
        const int lo = item.there.lo, hi = item.there.hi, sink_end = item.there.sink_end;
        const int32_t *const pages = item.pages;
        const int64_t k_at = p.io.k_off + (int64_t)item.h * D * 2, v_at = k_at + (p.io.v_off - p.io.k_off);
        item_read(k);
        int key = 0, page = -1;
        auto look_up = [&](int j) {  // one tile ahead of its copies
          key = (j < n_sink ? j : first_tile + j - n_sink) * kTileKeys + lw * 32 + lane;
          if (!(key < sink_end || (key >= lo && key < hi))) key = -1;
          page = key >= 0 ? pages[div_by(key, p.pools.page_size)] : -1;
        };
        if (n > 0) look_up(j0);
        for (int it = 0; it < n; ++it) {
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
          const uint32_t loaded = operands / 2;  // key tiles
          const int stage = loaded % kStages;
          const bool reuse = loaded >= kStages;
          const uint32_t freed = (loaded / kStages - 1) & 1;
#pragma unroll 1
          for (int which = 0; which < 2; ++which) {  // keys, then values
            uint64_t *full = which ? &bars.v_full[stage] : &bars.k_full[stage];
            ok = all(!reuse || wait_or_stop(which ? &bars.v_empty[stage] : &bars.k_empty[stage], freed));
            if (!ok) break;
            ++operands;
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
          if (!ok) break;
          if (warp == 8 && lane == 0 && it == (n > kClaimAhead ? n - kClaimAhead : 0)) mbar_arrive(&bars.wanted);
        }
        if (warp == 8 && lane == 0 && n == 0) mbar_arrive(&bars.wanted);
      }
      if (lane == 0) {
        bars.issued[lw] = operands;
        atomicSub(&bars.loaders, 1);
      }
      cp_async_wait_all();
    }
  } else {
    shrink_registers<kOthers>();
    const int role = __shfl_sync(0xffffffffu, warp, 0);
    if (role == kProducts) {
      // -------------------------------------------------------------- products
      // The copies are ordinary writes to shared memory: the fence of the warp that
      // issues the products (after the wait that orders them before it) lets the
      // tensor core see them.
      constexpr uint32_t desc_s = product_desc(kBf16, 128, kTileKeys, false), desc_o = product_desc(kBf16, 128, D, true);
      const uint32_t q_low = operand_low(smem_addr(q_smem), 16), k_low = operand_low(smem_addr(k_smem), 16);
      const uint32_t v_low = operand_low(smem_addr(v_smem), kTileKeys * 128);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      uint32_t used = 0, queries[2] = {0, 0}, weighed[2] = {0, 0};  // key tiles, query blocks, weight tiles
      // scores of tile t: queries of block q, keys of a stage
      auto scores = [&](int t, int q, int stage) {
        const uint32_t a = q_low + q * (Shape::kOperand >> 4), b = k_low + stage * (Shape::kOperand >> 4);
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
      auto values = [&](int t, int stage, uint32_t add) {
        const uint32_t b = v_low + stage * (Shape::kOperand >> 4), d = tm + 256 + t * 128, a = tm + t * 128;
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < kTileKeys / 16; ++e)  // weights lie over the scores that were held at a time
            mma_ts(d, a + (kQuantised ? e / 4 * 64 + e % 4 * 8 : e * 8), b + e * (16 * 128 >> 4), desc_o, e > 0 ? 1 : add);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t *bar) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      int turn = 0;  // query block of the next item that takes one
      auto keys_in = [&](uint32_t at) {
        wait(&bars.k_full[at % kStages], at / kStages);
        fence_proxy_async_smem();
      };
      auto values_in = [&](uint32_t at) {
        wait(&bars.v_full[at % kStages], at / kStages);
        fence_proxy_async_smem();
      };
      // weights of tile t times the values of a stage
      auto weigh = [&](int t, int stage, bool first) {
        wait(&bars.p_full[t], weighed[t]++);
        __syncwarp();
        tmem_fence_after();
        values(t, stage, !first);
      };
      for (int k = 0; item_there(k); ++k) {
        const int n = __shfl_sync(0xffffffffu, items[k % kItemSlots].n, 0);
        const int row_tiles = __shfl_sync(0xffffffffu, items[k % kItemSlots].group_tiles, 0);
        const int streams = __shfl_sync(0xffffffffu, items[k % kItemSlots].streams, 0);
        item_read(k);
        if (n == 0) continue;
        if (streams == 1) {
          wait(&bars.q_full[0], queries[0]++);
          wait(&bars.q_full[1], queries[1]++);
          auto queries_done = [&] {
            commit(&bars.q_empty[0]);
            commit(&bars.q_empty[1]);
          };
          keys_in(used);
          for (int t = 0; t < row_tiles; ++t) scores(t, t, used % kStages);
          commit(&bars.k_empty[used % kStages]);
          if (n == 1) queries_done();
          for (int it = 0; it < n; ++it) {
            const uint32_t at = used + it;
            const int stage = at % kStages, next = (at + 1) % kStages;
            values_in(at);
            if (it + 1 < n) {
              keys_in(at + 1);
              for (int t = 0; t < row_tiles; ++t) {
                weigh(t, stage, it == 0);
                if (t == row_tiles - 1) commit(&bars.v_empty[stage]);
                scores(t, t, next);
              }
              commit(&bars.k_empty[next]);
              if (it + 2 == n) queries_done();
            } else {
              for (int t = 0; t < row_tiles; ++t) {
                weigh(t, stage, it == 0);
                commit(&bars.o_full[t]);
              }
              commit(&bars.v_empty[stage]);
            }
          }
        } else {  // the same rows, every other key tile
          const int q = turn;
          turn ^= 1;
          if (q == 0) {
            wait(&bars.q_full[0], queries[0]++);
          } else {
            wait(&bars.q_full[1], queries[1]++);
          }
          keys_in(used);
          scores(0, q, used % kStages);
          commit(&bars.k_empty[used % kStages]);
          if (n > 1) {
            keys_in(used + 1);
            scores(1, q, (used + 1) % kStages);
            commit(&bars.k_empty[(used + 1) % kStages]);
          }
          if (n <= 2) commit(&bars.q_empty[q]);
          for (int it = 0; it < n; ++it) {
            const uint32_t at = used + it;
            const int t = it & 1, stage = at % kStages;
            values_in(at);
            weigh(t, stage, it < 2);
            commit(&bars.v_empty[stage]);
            if (it + 2 < n) {
              keys_in(at + 2);
              scores(t, q, (at + 2) % kStages);
              commit(&bars.k_empty[(at + 2) % kStages]);
              if (it + 3 == n) commit(&bars.q_empty[q]);
            } else {
              commit(&bars.o_full[t]);
            }
          }
        }
        used += n;
      }
    } else if (role == kProducts + 1) {
      // -------------------------------------------------------------- items
      if (lane == 0) {
        int block = (int)blockIdx.x;
        for (int k = 0;; ++k) {
          if (k >= kItemSlots && !wait_or_stop(&bars.item_empty[k % kItemSlots], k / kItemSlots - 1)) break;
          if (block >= 0) {
            find_item(p, block, &items[k % kItemSlots]);
          } else {
            items[k % kItemSlots].more = items[k % kItemSlots].n = 0;
          }
          mbar_arrive(&bars.item_full[k % kItemSlots]);
          if (!kTest || k == 0)
            *(volatile uint64_t *)&bars.deadline =
                global_timer_ns() + (kTest ? p.test_wait_ns : kTileWaitNs + items[k % kItemSlots].n * kTileStepNs);
          if (block < 0) break;
          if (!wait_or_stop(&bars.wanted, k)) break;  // the loads of this item near their end
          fence_proxy_async_smem();
          claim_block(&bars.claim, &bars.claimed);
          if (!wait_or_stop(&bars.claimed, k)) {  // the answer is on its way: the block stays until it is there
            tile_drain(&bars.claimed, k, global_timer_ns());
            break;
          }
          block = claimed_block(&bars.claim);
        }
      }
      __syncwarp();
    } else {
      // -------------------------------------------------------------- queries
      constexpr int kLanes = D / 8;
      const int at = (int)threadIdx.x - (kProducts + 2) * 32, c = at % kLanes;
      uint32_t filled[2] = {0, 0};
      int turn = 0;
      for (int k = 0; item_there(k); ++k) {
        int row0, rows;
        bool one;
        const char *q;
        {
          const TileItem &item = items[k % kItemSlots];
          row0 = item.row0, rows = item.rows, one = item.streams == 2;
          const bool none = item.n == 0;
          q = p.io.q + item.q_begin * p.io.q_stride + (int64_t)item.h * (int)p.io.group.d * (D * 2);
          item_read(k);
          if (none) continue;
        }
        const int block = one ? turn : 0;
        turn ^= one;
        // rows past the last keep what is there: nothing is made of them
        const int left = rows - row0, count = one ? left : left < kTileRows ? left : kTileRows;
        if (block == 0) {
          if (filled[0] > 0) wait(&bars.q_empty[0], filled[0] - 1);
          ++filled[0];
        }
        if (block == 1 || !one) {
          if (filled[1] > 0) wait(&bars.q_empty[1], filled[1] - 1);
          ++filled[1];
        }
        __syncwarp();
        // rows at / kLanes, + kStep, ...: (token, head) and address go along
        constexpr int kStep = 64 / kLanes;
        const int group = p.io.group.d, heads_on = kStep % group, tokens_on = kStep / group;
        const int64_t on = tokens_on * p.io.q_stride + heads_on * (D * 2), wrap = p.io.q_stride - group * (D * 2);
        int r = at / kLanes;
        const int i = div_by(row0 + r, p.io.group);
        int g = row0 + r - i * group;
        const char *src = q + i * p.io.q_stride + g * (D * 2) + c * 16;
        const uint32_t to = smem_addr(q_smem) + block * Shape::kOperand + (c >> 3) * (kTileKeys * 128);
#pragma unroll 8
        for (; r < count; r += kStep) {
          cp_async16(to + (r >> 7) * Shape::kOperand + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4), src);
          src += on;
          g += heads_on;
          if (g >= group) {
            g -= group;
            src += wrap;
          }
        }
        if (block == 0) mbar_arrive_after_copies(&bars.q_full[0]);
        if (block == 1 || !one) mbar_arrive_after_copies(&bars.q_full[1]);
      }
      cp_async_wait_all();
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kProducts) {
    if (*(volatile int *)&bars.gave_up) {  // what is in flight ends before the block and its tensor memory do
      if (elect_one()) mma_commit(&bars.drain);
      __syncwarp();
      const uint64_t t0 = global_timer_ns();
      tile_drain(&bars.drain, 0, t0);
      // the last use of every stage (of quantised rows the warps write the stages themselves)
      for (int w = 0; w < (kQuantised ? 0 : kLoadWarps); ++w) {
        const uint32_t values = bars.issued[w] / 2, keys = bars.issued[w] - values;
        for (uint32_t at = keys > kStages ? keys - kStages : 0; at < keys; ++at) tile_drain(&bars.k_full[at % kStages], at / kStages, t0);
        for (uint32_t at = values > kStages ? values - kStages : 0; at < values; ++at)
          tile_drain(&bars.v_full[at % kStages], at / kStages, t0);
      }
      __syncwarp();
    }
    tmem_free(tmem, 512);
  }
}

}  // namespace cpkv
