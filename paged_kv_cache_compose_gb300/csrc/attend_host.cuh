// The host side of the attention over paged rows: argument checks, workspace layout
// and the choice of passes, over rows of the element type or quantised ones.
#pragma once

#include "attend_join.cuh"
#include "attend_split_quantised.cuh"
#include "attend_unpack.cuh"

namespace cpkv {
namespace {

constexpr int kFewSeqs = 16;

// What both entry points are told of rows, heads and results.
struct HeadArgs {
  int dtype, q_heads, kv_heads, head_dim;
};

inline int check_heads(const HeadArgs &a) {
  if (a.dtype != CPKV_BF16 && a.dtype != CPKV_FP16) return CPKV_ERR_ARG;
  if (a.kv_heads < 1 || a.q_heads < 1 || a.q_heads % a.kv_heads != 0) return CPKV_ERR_ARG;
  if (a.head_dim != 64 && a.head_dim != 128) return CPKV_ERR_LIMIT;
  if (a.q_heads > 4096 || a.kv_heads > kSplitMaxGrid) return CPKV_ERR_LIMIT;
  return CPKV_OK;
}

// Where rows of the element type keep their keys and values.
inline int check_rows(const HeadArgs &a, int64_t row_bytes, int64_t k_off, int64_t v_off) {
  const int64_t bytes = (int64_t)a.kv_heads * a.head_dim * 2;
  if (k_off < 0 || v_off < 0 || k_off % 16 != 0 || v_off % 16 != 0) return CPKV_ERR_ARG;
  if (k_off + bytes > row_bytes || v_off + bytes > row_bytes) return CPKV_ERR_ARG;
  return CPKV_OK;
}

inline int fill_io(AttendIo *io, const HeadArgs &a, const void *q, int64_t q_stride, void *out, int64_t out_stride, float *lse,
            float scale, int64_t k_off, int64_t v_off) {
  const int64_t width = (int64_t)a.q_heads * a.head_dim;
  if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out)) return CPKV_ERR_ARG;
  if (q_stride < width || out_stride < width || q_stride % 8 != 0 || out_stride % 8 != 0) return CPKV_ERR_ARG;
  if (!(scale > 0.f && scale < INFINITY)) return CPKV_ERR_ARG;
  io->q = static_cast<const char *>(q);
  io->out = static_cast<char *>(out);
  io->lse = lse;
  io->q_stride = q_stride * 2;
  io->out_stride = out_stride * 2;
  io->q_heads = a.q_heads;
  io->kv_heads = a.kv_heads;
  io->group = fast_div((uint32_t)(a.q_heads / a.kv_heads));
  io->scale_log2 = scale * kLog2e;
  io->k_off = k_off;
  io->v_off = v_off;
  return CPKV_OK;
}

inline int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

// Bounds of a split pass, from host lengths.
struct SplitBounds {
  int64_t units = 0, max_tiles = 0;  // of all sequences, of one
  int grid_cap = 1;

  void add(int64_t nq, int64_t max_kv, int window, int sinks) {
    int64_t tiles = ceil_div(max_kv, kSplitTile);
    if (window > 0) tiles = std::min<int64_t>(tiles, ceil_div((int64_t)sinks, kSplitTile) + ((int64_t)window + nq) / kSplitTile + 2);
    units += nq > 0 ? tiles : 0;
    max_tiles = std::max<int64_t>(max_tiles, tiles);
  }
  int finish(int kv_heads) {
    if (units > INT32_MAX) return CPKV_ERR_LIMIT;
    grid_cap = kv_heads * (int)std::min<int64_t>(kSplitMaxGrid / kv_heads, units > 0 ? units : 1);
    return CPKV_OK;
  }
  int64_t slots(int64_t count, int kv_heads, bool direct) const { return 2 * (int64_t)grid_cap + (direct ? 0 : count * kv_heads); }
  int64_t bytes(int64_t count, int kv_heads, int head_dim, bool direct) const {
    const int64_t n = slots(count, kv_heads, direct) * kSplitRows;
    return round_up((count + 1) * 4, 256) + round_up(n * 8, 256) + round_up(n * head_dim * 4, 256);
  }
  SplitSpace space(char *at, int64_t count, int kv_heads, bool direct) const {
    SplitSpace s;
    s.cum = reinterpret_cast<int32_t *>(at);
    at += round_up((count + 1) * 4, 256);
    s.ml = reinterpret_cast<float *>(at);
    at += round_up(slots(count, kv_heads, direct) * kSplitRows * 8, 256);
    s.o = reinterpret_cast<float *>(at);
    s.grid = grid_cap;
    return s;
  }
};

// Bounds and splits of a tile pass: ragged sequences, and (of a shared call) the
// suffixes, of one query each.
struct TileBounds {
  int64_t tokens = 0, tiles = 0, max_rows = 0, max_keys = 0;
  int64_t singles = 0, single_keys = 0, single_tiles = 0, group = 1;
  int splits = 1, single_splits = 1;

  // Beginning and end of an item, and the joining of parts, in 128-key steps (about
  // 4 us and 6 us against 1.4 us a step, measured).
  static constexpr int64_t kItemSteps = 3, kJoinSteps = 4;

  void add(int64_t nq, int64_t max_kv, int of_group, int window, int sinks) {
    int64_t seen = max_kv;
    if (window > 0) seen = std::min<int64_t>(seen, (int64_t)window + kTileRows / of_group + sinks);
    group = of_group;
    tiles += ceil_div(nq * group, kTileRows);
    tokens += nq;
    max_rows = std::max<int64_t>(max_rows, nq * group);
    max_keys = std::max<int64_t>(max_keys, seen);
  }
  void add_singles(int64_t count, int64_t max_kv) {
    singles = count;
    single_keys = max_kv;
    single_tiles = ceil_div(group, kTileRows);
  }
  // Steps over keys: two streams take the key tiles of at most 128 rows two at a time.
  static int64_t steps(int64_t keys, int64_t rows) { return ceil_div(keys, rows <= 128 ? 2 * kTileKeys : kTileKeys); }
  int check(int kv_heads) const {
    const int64_t items = tiles * kv_heads, single_items = singles * single_tiles * kv_heads;
    if (items > INT32_MAX / 1024 || single_items > INT32_MAX / 1024 || tokens > INT32_MAX) return CPKV_ERR_LIMIT;
    return CPKV_OK;
  }
  // How many parts an item's keys are cut into: the count whose rounds of blocks over
  // the SMs come to the fewest steps.  Of keys that are converted on the way a tile is a step,
  // whoever multiplies it, and the fewest steps are taken however close the next: 12 requests of 160
  // rows on 8192 keys, 8 heads, 101 us so and 133 with the rule of plain rows, one of 120 on 20000 18.8 and 20.8.
  int finish(int kv_heads, int head_dim, bool converts) {
    const int64_t items = tiles * kv_heads, sms = device_sm_count();
    const int64_t all = converts ? ceil_div(max_keys, kTileKeys) : steps(max_keys, max_rows);
    int64_t best = INT64_MAX / 16;
    for (int64_t n = 1; n <= std::min<int64_t>(std::max<int64_t>(all / 2, 1), sms) && items > 0; ++n) {
      if (n > 1 && items * n > 4 * sms) break;
      // in 32nds of a step; a part of 256 rows of 128 written and read again is about one
      const int64_t cost = 32 * ceil_div(items * n, sms) * (ceil_div(all, n) + kItemSteps) +
                           (n > 1 ? 32 * kJoinSteps + items * n * head_dim / 128 : 0);
      if (converts ? cost < best : 10 * cost < 9 * best) {  // for a tenth or more
        best = cost;
        splits = (int)n;
      }
    }
    return check(kv_heads);
  }
  // Prefixes and suffixes of a shared call: as few parts as leave no item longer than
  // the SMs' even share of all work (a suffix counted at half its bound and a step).
  // 48 requests of three prefixes of about 9000: 41.3 us so, 44.5 with items of half that
  // length, 49.2 of one and a half; 256 requests on one of 65536: 556, 572 and 555 us.
  int finish_shared(int kv_heads) {
    const int64_t items = tiles * kv_heads, single_items = singles * single_tiles * kv_heads, sms = device_sm_count();
    const int64_t all = steps(max_keys, max_rows), of_single = steps(single_keys, group);
    const int64_t share = ceil_div(items * all + single_items * (ceil_div(of_single, 2) + 1), sms);
    const int64_t most = std::max<int64_t>(share, 4);
    splits = (int)std::min<int64_t>(std::max<int64_t>(ceil_div(all, most), 1), sms);
    single_splits = (int)std::min<int64_t>(std::max<int64_t>(ceil_div(of_single, most), 1), sms);
    return check(kv_heads);
  }
  int64_t blocks(int kv_heads) const { return kv_heads * (tiles * splits + singles * single_tiles * single_splits); }
  int64_t ragged_rows(int kv_heads) const { return tiles * kv_heads * splits * kTileRows; }
  int64_t rows(int kv_heads) const {
    return ragged_rows(kv_heads) + singles * single_tiles * kv_heads * single_splits * std::min<int64_t>(group, kTileRows) + kTileRows;
  }
  int64_t bytes(int kv_heads, int head_dim, bool direct) const {
    if (direct && splits == 1) return 0;
    return kPartAlign + round_up(rows(kv_heads) * 8, 256) + round_up(rows(kv_heads) * head_dim * 4, 256);
  }
  // The parts' values go out 32 bytes at a time, and a caller's workspace may begin at
  // any multiple of 16: bytes() counts the room for the step to the next 32.
  static constexpr int64_t kPartAlign = 32;
  TileSpace space(char *at, int kv_heads) const {
    at += -reinterpret_cast<uintptr_t>(at) & (kPartAlign - 1);
    TileSpace s;
    s.ml = reinterpret_cast<float *>(at);
    s.o = reinterpret_cast<float *>(at + round_up(rows(kv_heads) * 8, 256));
    s.splits = splits;
    s.single_splits = single_splits;
    s.items = (int)(tiles * kv_heads);
    s.single_tiles = (int)single_tiles;
    s.single_row = ragged_rows(kv_heads);
    s.by_heads = fast_div((uint32_t)kv_heads);
    s.by_splits = fast_div((uint32_t)splits);
    s.by_single_splits = fast_div((uint32_t)single_splits);
    s.by_single_tiles = fast_div((uint32_t)std::max<int64_t>(single_tiles, 1));
    return s;
  }
};

// Which kernel reads the keys: the split kernel takes 16 packed rows at a time
// and reads the keys again for each 16, the tile kernel takes 256.  64 requests of
// 2048 keys, 8 heads of 128: at 16 rows 88 us with the split kernel and 95 with the
// tile kernel, at 24 rows 160 and 103 us.
inline bool few_rows(int64_t max_rows) { return max_rows <= kSplitRows; }

// Quantised rows that a tile pass brings to the element type beforehand (attend_unpack.cuh):
// where a call's sequences come to kUnpackTiles row tiles or more on the average, and the dense rows, of
// all of them at the bound of the lengths, fit kUnpackMost (the passes over the rows themselves need next to no
// memory).  5 requests of up to
// 16384 keys, 32 heads of 128 on 8, beforehand and on the way: one row tile 120 and 99 us, two 138 and
// 123, three 217 and 237, four 202 and 203, six 238 and 269, eight 287 and 338; 32 requests: two
// 801 and 667, four 1162 and 1179.  That is of equal requests; in a ragged call the average may read rows
// back that few queries see: 4096 tokens beside 15 single ones, all on 16384 keys, 1092 and 1104 us (1 GiB of rows), on
// 4096 keys 227 and 199, the 4096 on as many and the others on 32768 keys 927 and 475.
struct UnpackBounds {
  int64_t pages = 0, stride = 0;
  int sequences = 0;

  static int64_t pages_of(int64_t nq, int64_t max_kv, int window, int sinks) {
    const int64_t all = ceil_div(max_kv, kDensePage);
    if (nq == 0) return 0;
    if (window == 0) return all;
    return std::min<int64_t>(all, ceil_div((int64_t)sinks, kDensePage) + ((int64_t)window + nq) / kDensePage + 2);
  }
  void add(int64_t nq, int64_t max_kv, int window, int sinks) {
    pages += pages_of(nq, max_kv, window, sinks);
    sequences += nq > 0;
    stride = ceil_div(max_kv, kDensePage);
  }
  static int64_t row_bytes(int kv_heads, int head_dim) { return (int64_t)kv_heads * head_dim * 4; }
  int64_t table_bytes(int64_t count) const { return round_up(count * stride * 4, 256); }
  int64_t bytes(int64_t count, int kv_heads, int head_dim) const {
    return table_bytes(count) + pages * kDensePage * row_bytes(kv_heads, head_dim) + 256;
  }
};

constexpr int64_t kUnpackTiles = 4, kUnpackMost = (int64_t)1 << 32;

// How a call is done, from host lengths alone.
struct WindowPlan {
  SplitBounds split;
  TileBounds tile;
  UnpackBounds unpack;
  bool few = true, whole = false, unpacks = false;
  int64_t tokens = 0, bytes = 0, pass_bytes = 0;  // of the workspace: in all, of the passes alone
};

// A window that no request's keys reach past is none: positions less it stay in 32 bits,
// also below 0 (a request shorter than its queries).
inline int clamp_window(int window, int64_t max_kv) { return window >= max_kv ? 0 : window; }

inline int window_plan(WindowPlan *w, const HeadArgs &a, bool quantised, int B, const int32_t *h_q_lens, int64_t max_kv, int window, int sinks) {
  const int group = a.q_heads / a.kv_heads;
  for (int s = 0; s < B; ++s) {
    const int64_t nq = h_q_lens == nullptr ? 1 : h_q_lens[s];
    if (nq < 0) return CPKV_ERR_ARG;
    w->split.add(nq, max_kv, window, sinks);
    w->tile.add(nq, max_kv, group, window, sinks);
    w->unpack.add(nq, max_kv, window, sinks);
  }
  w->few = few_rows(w->tile.max_rows);
  w->tokens = w->tile.tokens;
  bool uniform = B > 0;
  for (int s = 1; s < B && h_q_lens != nullptr; ++s) uniform &= h_q_lens[s] == h_q_lens[0];
  // A block takes a whole sequence of few rows when none has more units of keys
  // than kWholeUnits and there are no more of them than SMs: the units one after the other then
  // cost less than joining parts does (4 requests, 8 heads of 128: 384 keys in 10.3 us
  // where parts take 12.3, 512 keys in 12.3 either way, 1024 in 20.5 where parts take
  // 13.4), and no more blocks wait than lines would have (64 requests of 384 keys: 36 us
  // with whole sequences, 26 with parts).
  w->whole = w->few && uniform && w->split.max_tiles <= kWholeUnits &&
             (int64_t)B * a.kv_heads <= device_sm_count();
  w->unpacks = quantised && !w->few && w->unpack.pages > 0 && w->tile.tiles >= kUnpackTiles * w->unpack.sequences &&
               w->unpack.bytes(B, a.kv_heads, a.head_dim) <= kUnpackMost;
  const int rc = w->few ? w->split.finish(a.kv_heads) : w->tile.finish(a.kv_heads, a.head_dim, quantised && !w->unpacks);
  w->bytes = w->whole ? 0
             : w->few ? w->split.bytes(B, a.kv_heads, a.head_dim, true)
                      : w->tile.bytes(a.kv_heads, a.head_dim, true);
  w->pass_bytes = round_up(w->bytes, 256);
  if (w->unpacks) w->bytes = w->pass_bytes + w->unpack.bytes(B, a.kv_heads, a.head_dim);
  return rc;
}

struct SharedPlan {
  SplitBounds split;  // prefixes and suffixes when rows are few
  TileBounds tile;    // and when they are many
  bool few = true, mixed = false;  // mixed: prefixes by the tile pass, suffixes by the split pass
  int64_t prefix_pages = 0, bytes = 0, split_at = 0;  // split_at: of a mixed call, where the split pass's workspace begins
};

// Quantised suffixes beside prefixes of many rows go to the split pass where they come to two key tiles
// or more for each SM: a tile pass would convert and multiply them for 128 rows of which few are real,
// against 2 us for another kernel.  32 heads of 128 on 8, a prefix of 16384: 32 requests with
// suffixes of up to 1024 in 37 us, 53 in one pass; 16 with up to 64, which is below, 37.0 and 36.6; a
// prefix of 1024 and 32 suffixes of up to 32, 28.8 and 27.1.
inline bool mixes(SharedPlan &w, const HeadArgs &a, bool quantised, int B, int64_t max_suffix) {
  if (!quantised || !few_rows(a.q_heads / a.kv_heads)) return false;
  if ((int64_t)B * a.kv_heads * ceil_div(max_suffix, kTileKeys) < 2 * device_sm_count()) return false;
  for (int b = 0; b < B; ++b) w.split.add(1, max_suffix, 0, 0);
  return w.split.finish(a.kv_heads) == CPKV_OK;
}

inline int shared_plan(SharedPlan *w, const HeadArgs &a, bool quantised, int B, int n_groups, const int32_t *h_group_sizes,
                const int32_t *h_prefix_lens, int page_size, int64_t max_suffix) {
  const int group = a.q_heads / a.kv_heads;
  int64_t sum = 0;
  for (int g = 0; g < n_groups; ++g) {
    if (h_group_sizes[g] < 0 || h_prefix_lens[g] < 0) return CPKV_ERR_ARG;
    if (page_size > 0 && h_prefix_lens[g] % page_size != 0) return CPKV_ERR_UNALIGNED_PREFIX;
    if (h_prefix_lens[g] > INT32_MAX / 2) return CPKV_ERR_LIMIT;
    w->tile.add(h_group_sizes[g], h_prefix_lens[g], group, 0, 0);
    sum += h_group_sizes[g];
    if (page_size > 0) w->prefix_pages += h_prefix_lens[g] / page_size;
  }
  if (sum != B) return CPKV_ERR_ARG;
  if (w->prefix_pages > INT32_MAX) return CPKV_ERR_LIMIT;
  w->few = few_rows(w->tile.max_rows);
  int rc;
  if (w->few) {
    for (int g = 0; g < n_groups; ++g) w->split.add(h_group_sizes[g], h_prefix_lens[g], 0, 0);
    for (int b = 0; b < B; ++b) w->split.add(1, max_suffix, 0, 0);
    rc = w->split.finish(a.kv_heads);
    w->bytes = w->split.bytes(n_groups + B, a.kv_heads, a.head_dim, false);
  } else if (mixes(*w, a, quantised, B, max_suffix)) {
    w->mixed = true;
    rc = w->tile.finish(a.kv_heads, a.head_dim, false);  // (fewer parts leave SMs to the split pass: 39.0 us, 43.3 counted as above)
    w->split_at = round_up(w->tile.bytes(a.kv_heads, a.head_dim, false), 256);
    w->bytes = w->split_at + w->split.bytes(B, a.kv_heads, a.head_dim, false);
  } else {
    w->tile.add_singles(B, max_suffix);
    rc = w->tile.finish_shared(a.kv_heads);
    w->bytes = w->tile.bytes(a.kv_heads, a.head_dim, false);
  }
  return rc;
}

// Which split kernel and shape.
struct Plain {};
template <int kBlocks8>
struct Quantised {};
template <typename T, int D, SplitMode kMode, typename S, typename Rows>
struct SplitPass {
  using Shape = SplitShape<D, kMode>;
  static constexpr auto kernel = attend_split_kernel<T, D, S, kMode>;
};
template <typename T, int D, SplitMode kMode, typename S, int kBlocks8>
struct SplitPass<T, D, kMode, S, Quantised<kBlocks8>> {
  using Shape = SplitShapeQ<D, kMode, kBlocks8>;
  static constexpr auto kernel = attend_split_quantised_kernel<T, D, S, kMode, kBlocks8>;
};

template <typename F>
int for_type_and_dim(const HeadArgs &a, F f) {
  if (a.dtype == CPKV_BF16) {
    return a.head_dim == 128 ? f(__nv_bfloat16(), std::integral_constant<int, 128>())
                             : f(__nv_bfloat16(), std::integral_constant<int, 64>());
  }
  return a.head_dim == 128 ? f(__half(), std::integral_constant<int, 128>())
                           : f(__half(), std::integral_constant<int, 64>());
}

// A block takes a whole sequence unless the mode is kLine.
template <typename T, int D, SplitMode kMode, typename Rows, typename S>
int split_pass_of(SplitParams<S> *p, const SplitBounds &b, bool dependent, cudaStream_t stream) {
  using Pass = SplitPass<T, D, kMode, S, Rows>;
  using Shape = typename Pass::Shape;
  const int smem = Shape::kSmem + (kMode == kLine ? (p->seqs.count + 1) * 4 : 0);
  auto kernel = Pass::kernel;
  const int rc = ensure_dynamic_smem((const void *)kernel, Shape::kSmem + (kMode == kLine ? (2 * CPKV_MAX_BATCH + 1) * 4 : 0));
  if (rc != CPKV_OK) return rc;
  int64_t blocks = (int64_t)p->seqs.count * p->io.kv_heads;
  if (kMode == kLine) {  // as many blocks for every head as stay resident together
    const int heads = p->io.kv_heads, resident = persistent_grid((const void *)kernel, kSplitWarps * 32, smem, 8, b.grid_cap);
    blocks = p->space.grid = std::max(resident / heads, 1) * heads;
  }
  if (blocks > INT32_MAX) return CPKV_ERR_LIMIT;
  return launch_kernel(kernel, dim3((unsigned)blocks), dim3(kSplitWarps * 32), smem, dependent, stream, *p);
}

// max_rows: of a sequence.  dependent: may begin while the kernel before it runs (quantised rows).
template <typename T, int D, SplitMode kMode, bool kQuantised, typename S>
int split_pass(SplitParams<S> *p, const SplitBounds &b, int64_t max_rows, cudaStream_t stream, bool dependent = false) {
  if constexpr (!kQuantised) {
    return split_pass_of<T, D, kMode, Plain>(p, b, false, stream);
  } else {
    return max_rows <= 8 ? split_pass_of<T, D, kMode, Quantised<1>>(p, b, dependent, stream)
                         : split_pass_of<T, D, kMode, Quantised<2>>(p, b, dependent, stream);
  }
}

template <typename S>
SplitSource<S> source_of(const SplitParams<S> &p) {
  SplitSource<S> s;
  s.seqs = p.seqs;
  s.space = p.space;
  s.direct = p.direct;
  return s;
}

// cuTensorMapEncodeTiled, looked up once; null where the driver has none.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
  static const EncodeTiled found = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess) {
      (void)cudaGetLastError();
      return (EncodeTiled) nullptr;
    }
    return how == cudaDriverEntryPointSuccess ? (EncodeTiled)f : (EncodeTiled) nullptr;
  }();
  return found;
}

// TMA maps of the pools: [rows][elements], boxes of `box` rows by 64 elements in
// the 128-byte swizzle of the kernel's shared memory.  Pages of 16 rows or a
// multiple have them; others (and more than kTileMaps pools) leave box_rows 0,
// and the kernel copies key by key.
template <typename S>
void fill_maps(TileParams<S> *p) {
  const uint32_t ps = p->pools.page_size.d;
  p->box_rows = 0;
  if (ps % 16 != 0 || p->pools.cp.d > kTileMaps || encode_tiled() == nullptr) return;
  const cuuint32_t box[2] = {64, ps % 32 == 0 ? 32u : 16u}, steps[2] = {1, 1};
  for (uint32_t r = 0; r < p->pools.cp.d; ++r) {
    const int64_t rows = (int64_t)p->pools.cap[r] * ps;
    if (rows == 0) continue;  // no page of it is valid
    if (rows > INT32_MAX) return;
    const cuuint64_t dims[2] = {(cuuint64_t)p->pools.row_bytes / 2, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)p->pools.row_bytes};
    if (encode_tiled()(&p->maps[r], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p->pools.pool[r], dims, strides, box, steps,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return;
  }
  p->box_rows = (int)box[1];
}

template <bool kQuantised, typename S>
void fill_tiles(TileParams<S> *p, const S &seqs, int ragged, const PagedPools &pools, const AttendIo &io,
                const TileBounds &b, char *workspace, bool direct) {
  p->seqs = seqs;
  p->pools = pools;
  p->io = io;
  p->space = b.space(workspace, io.kv_heads);
  p->direct = direct && b.splits == 1;
  p->wide_out = (reinterpret_cast<uintptr_t>(io.out) & 31) == 0 && io.out_stride % 32 == 0;
  if (!kQuantised) fill_maps(p);
  const int group = io.group.d;
  for (int s = 0; s < ragged; ++s)
    p->cu_tiles[s + 1] = p->cu_tiles[s] + (int)ceil_div((int64_t)(seqs.cu_q[s + 1] - seqs.cu_q[s]) * group, kTileRows);
}

template <typename T, int D, bool kQuantised, bool kTest = false, typename S>
int tile_pass(const TileParams<S> &p, const TileBounds &b, cudaStream_t stream) {
  auto kernel = attend_tile_kernel<T, D, S, kTest, kQuantised>;
  const int rc = ensure_dynamic_smem((const void *)kernel, TileShape<D, kQuantised>::kSmem);
  if (rc != CPKV_OK) return rc;
  const int64_t grid = b.blocks(p.io.kv_heads);
  if (grid > INT32_MAX) return CPKV_ERR_LIMIT;
  return launch_kernel(kernel, dim3((unsigned)grid), dim3(tile_threads(kQuantised)), TileShape<D, kQuantised>::kSmem, false, stream, p);
}

template <typename S>
TileSource<S> source_of(const TileParams<S> &p) {
  TileSource<S> s;
  s.seqs = p.seqs;
  s.space = p.space;
  std::copy(p.cu_tiles, p.cu_tiles + S::kArray + 1, s.cu_tiles);
  return s;
}

// Four warps a row while rows are too few to fill the SMs with a warp each: 32 rows
// of 8192 keys take 18.0 us with four and 22.6 with one, 8192 rows of 1024 keys 252 us
// with four and 158 with one (both with the pass before them).
template <typename T, int D, typename Source>
int join_pass(const Source &source, const AttendIo &io, int64_t rows, cudaStream_t stream) {
  JoinParams<Source> p = {};
  p.source = source;
  p.io = io;
  p.rows = rows;
  const bool wide = rows <= (int64_t)device_sm_count() * 16;
  const int64_t blocks = wide ? rows : ceil_div(rows, 4);
  if (blocks > INT32_MAX) return CPKV_ERR_LIMIT;
  auto kernel = wide ? attend_join_kernel<T, D, Source, 4> : attend_join_kernel<T, D, Source, 1>;
  return launch_kernel(kernel, dim3((unsigned)blocks), dim3(128), 0, true, stream, p);
}

template <bool kQuantised, int N>
int attend_window(const HeadArgs &heads, const Seqs<N> &seqs, const PagedPools &pools, const AttendIo &io,
                  const WindowPlan &plan, char *workspace, cudaStream_t stream) {
  const int64_t rows = plan.tokens * heads.q_heads;
  if (plan.few) {
    SplitParams<Seqs<N>> p = {};
    p.seqs = seqs;
    p.pools = pools;
    p.io = io;
    p.direct = 1;
    if (plan.whole) {
      return for_type_and_dim(heads, [&](auto t, auto d) {
        return split_pass<decltype(t), decltype(d)::value, kFewKeys, kQuantised>(&p, plan.split, plan.tile.max_rows, stream);
      });
    }
    p.space = plan.split.space(workspace, seqs.count, heads.kv_heads, true);
    return for_type_and_dim(heads, [&](auto t, auto d) {
      using T = decltype(t);
      constexpr int D = decltype(d)::value;
      const int rc = split_pass<T, D, kLine, kQuantised>(&p, plan.split, plan.tile.max_rows, stream);
      return rc != CPKV_OK ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
    });
  }
  TileParams<Seqs<N>> p = {};
  fill_tiles<kQuantised>(&p, seqs, seqs.count, pools, io, plan.tile, workspace, true);
  return for_type_and_dim(heads, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    const int rc = tile_pass<T, D, kQuantised>(p, plan.tile, stream);
    return rc != CPKV_OK || p.direct ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
  });
}

// Quantised prefixes in a tile pass; suffixes in a split pass, whose blocks take the SMs as the
// tile pass leaves them; both joined.
template <int N>
int attend_mixed(const HeadArgs &heads, const SharedSeqs<N> &seqs, const PagedPools &pools, const AttendIo &io,
                 const SharedPlan &plan, char *workspace, cudaStream_t stream) {
  const int64_t rows = (int64_t)(seqs.count - seqs.groups) * heads.q_heads;
  TileParams<SharedSeqs<N>> t = {};
  fill_tiles<true>(&t, seqs, seqs.groups, pools, io, plan.tile, workspace, false);
  using One = SharedSeqs<kFewSeqs>;  // the requests alone
  SplitParams<One> p = {};
  p.seqs.table = seqs.table;
  p.seqs.suffix_lens = seqs.suffix_lens;
  p.seqs.stride = seqs.stride;
  p.seqs.status = seqs.status;
  p.seqs.suffix_cap = seqs.suffix_cap;
  p.seqs.count = seqs.count - seqs.groups;
  p.pools = pools;
  p.io = io;
  p.space = plan.split.space(workspace + plan.split_at, p.seqs.count, heads.kv_heads, false);
  return for_type_and_dim(heads, [&](auto type, auto dim) {
    using T = decltype(type);
    constexpr int D = decltype(dim)::value;
    int rc = tile_pass<T, D, true>(t, plan.tile, stream);
    if (rc != CPKV_OK) return rc;
    rc = split_pass<T, D, kLine, true>(&p, plan.split, io.group.d, stream, true);
    if (rc != CPKV_OK) return rc;
    return join_pass<T, D>(MixedSource<SharedSeqs<N>, One>{source_of(t), source_of(p)}, io, rows, stream);
  });
}

// Prefixes and suffixes in one pass, joined (quantised ones beside many rows in two).
template <bool kQuantised, int N>
int attend_shared(const HeadArgs &heads, const SharedSeqs<N> &seqs, const PagedPools &pools, const AttendIo &io,
                  const SharedPlan &plan, char *workspace, cudaStream_t stream) {
  const int64_t rows = (int64_t)(seqs.count - seqs.groups) * heads.q_heads;
  if (plan.few) {
    SplitParams<SharedSeqs<N>> p = {};
    p.seqs = seqs;
    p.pools = pools;
    p.io = io;
    p.space = plan.split.space(workspace, seqs.count, heads.kv_heads, false);
    return for_type_and_dim(heads, [&](auto t, auto d) {
      using T = decltype(t);
      constexpr int D = decltype(d)::value;
      const int rc = split_pass<T, D, kLine, kQuantised>(&p, plan.split, plan.tile.max_rows, stream);
      return rc != CPKV_OK ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
    });
  }
  if constexpr (kQuantised) {
    if (plan.mixed) return attend_mixed(heads, seqs, pools, io, plan, workspace, stream);
  }
  TileParams<SharedSeqs<N>> p = {};
  fill_tiles<kQuantised>(&p, seqs, seqs.groups, pools, io, plan.tile, workspace, false);
  return for_type_and_dim(heads, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    const int rc = tile_pass<T, D, kQuantised>(p, plan.tile, stream);
    return rc != CPKV_OK ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
  });
}

// What the entry points are told, beside the heads; `row` of quantised rows (the offsets come from it).
struct RowArgs {
  int page_size, cp_size;
  int64_t row_bytes, key_offset, value_offset;
  const cpkv_quantised_row *row;
  const void *const *h_pools;
  const int64_t *h_pool_cap_pages;
  int flags;
};

struct ResultArgs {
  const void *d_q;
  int64_t q_stride;
  float scale;
  void *d_out;
  int64_t out_stride;
  float *d_lse;
  void *d_workspace;
  int64_t workspace_bytes;
  int32_t *d_status;
  cudaStream_t stream;
};

template <bool kQuantised>
int open_rows(PagedPools *pools, const HeadArgs &heads, const RowArgs &a) {
  const int rc = paged_pools(pools, a.page_size, a.cp_size, a.row_bytes, a.h_pools, a.h_pool_cap_pages, a.flags);
  return rc != CPKV_OK || kQuantised ? rc : check_rows(heads, a.row_bytes, a.key_offset, a.value_offset);
}

template <bool kQuantised>
int fill_io(AttendIo *io, const HeadArgs &heads, const RowArgs &rows, const ResultArgs &r) {
  if (kQuantised) {
    io->ks_off = rows.row->key_scale_offset;
    io->vs_off = rows.row->value_scale_offset;
  }
  return fill_io(io, heads, r.d_q, r.q_stride, r.d_out, r.out_stride, r.d_lse, r.scale, rows.key_offset, rows.value_offset);
}

// The heads and rows of a quantised call: rows whose keys and values are as wide as the heads.
inline int quantised_rows(HeadArgs *heads, RowArgs *rows, int dtype, int q_heads, const cpkv_quantised_row *row) {
  const int rc = check_quantised_row(row);
  if (rc != CPKV_OK) return rc;
  if (row->keep_keys || row->key_dim != row->value_dim) return CPKV_ERR_ARG;
  *heads = HeadArgs{dtype, q_heads, row->kv_heads, row->key_dim};
  rows->row = row;
  rows->row_bytes = row->row_bytes;
  rows->key_offset = row->key_offset;
  rows->value_offset = row->value_offset;
  return CPKV_OK;
}

struct WindowCall {
  int B;
  const int32_t *h_q_lens;
  int64_t max_kv_len;
  const int32_t *d_page_table;
  int64_t table_stride;
  const int32_t *d_kv_lens;
  int64_t num_tokens;
  int window, sinks;
};

// The rows that the queries see into dense pages, then the call over those.
template <int N>
int unpacked_call(const HeadArgs &heads, const Seqs<N> &s, const PagedPools &pools, const AttendIo &io, const WindowPlan &plan,
                  const WindowCall &c, const ResultArgs &r) {
  char *at = static_cast<char *>(r.d_workspace) + plan.pass_bytes;
  at += -reinterpret_cast<uintptr_t>(at) & 255;
  UnpackParams<Seqs<N>> p = {};
  p.seqs = s;
  p.pools = pools;
  p.io = io;
  p.table = reinterpret_cast<int32_t *>(at);
  p.table_stride = plan.unpack.stride;
  p.rows = at + plan.unpack.table_bytes(c.B);
  for (int b = 0; b < c.B; ++b)
    p.cu_pages[b + 1] = p.cu_pages[b] + (int)UnpackBounds::pages_of(c.h_q_lens == nullptr ? 1 : c.h_q_lens[b], c.max_kv_len, s.window, s.sinks);
  const int64_t blocks = plan.unpack.pages * (kDensePage / kUnpackRows), row_bytes = UnpackBounds::row_bytes(heads.kv_heads, heads.head_dim);
  if (blocks > INT32_MAX) return CPKV_ERR_LIMIT;
  int rc = for_type_and_dim(heads, [&](auto t, auto d) {
    return launch_kernel(unpack_kernel<decltype(t), decltype(d)::value, Seqs<N>>, dim3((unsigned)blocks), dim3(kUnpackRows * 32), 0, false, r.stream, p);
  });
  if (rc != CPKV_OK) return rc;
  const void *const rows = p.rows;
  const int64_t cap = plan.unpack.pages;
  return cpkv_attend_window(c.B, kDensePage, 1, heads.dtype, heads.q_heads, heads.kv_heads, heads.head_dim, row_bytes, 0, row_bytes / 2,
                            c.h_q_lens, c.max_kv_len, &rows, &cap, p.table, p.table_stride, c.d_kv_lens, c.num_tokens, r.d_q, r.q_stride,
                            r.scale, c.window, c.sinks, r.d_out, r.out_stride, r.d_lse, r.d_workspace, plan.pass_bytes,
                            CPKV_DENSE_PAGES, r.d_status, (cpkv_stream_t)r.stream);
}

template <bool kQuantised>
int window_call(const HeadArgs &heads, const RowArgs &rows, const WindowCall &c, const ResultArgs &r) {
  const int B = c.B;
  if (B < 0 || c.max_kv_len < 0 || c.window < 0 || c.sinks < 0 || (rows.flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || c.max_kv_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  PagedPools pools = {};
  rc = open_rows<kQuantised>(&pools, heads, rows);
  if (rc != CPKV_OK) return rc;
  if (c.table_stride < 0 || c.max_kv_len > c.table_stride * rows.page_size) return CPKV_ERR_CAPACITY;
  const int window = clamp_window(c.window, c.max_kv_len);
  WindowPlan plan;
  rc = window_plan(&plan, heads, kQuantised, B, c.h_q_lens, c.max_kv_len, window, c.sinks);
  if (rc != CPKV_OK) return rc;
  if (plan.tokens != c.num_tokens) return CPKV_ERR_ARG;
  if (plan.tokens == 0) return CPKV_OK;
  if (c.d_kv_lens == nullptr || r.d_status == nullptr || (c.max_kv_len > 0 && c.d_page_table == nullptr)) return CPKV_ERR_ARG;
  AttendIo io = {};
  rc = fill_io<kQuantised>(&io, heads, rows, r);
  if (rc != CPKV_OK) return rc;
  if (r.workspace_bytes < plan.bytes) return CPKV_ERR_CAPACITY;
  if (plan.bytes > 0 && (r.d_workspace == nullptr || !aligned16(r.d_workspace))) return CPKV_ERR_ARG;
  // one query length for all needs no lengths in the kernel's block (the tile kernel goes by them)
  bool uniform = plan.few;
  for (int b = 1; b < B && c.h_q_lens != nullptr; ++b) uniform &= c.h_q_lens[b] == c.h_q_lens[0];
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Seqs<N> s = {};
    s.kv_lens = c.d_kv_lens;
    s.table = c.d_page_table;
    s.stride = c.table_stride;
    s.status = r.d_status;
    s.count = B;
    s.kv_cap = (int)c.max_kv_len;
    s.window = window;
    s.sinks = c.sinks;
    if (uniform) {
      s.uniform_q = c.h_q_lens == nullptr ? 1 : c.h_q_lens[0];
    } else {
      for (int b = 0; b < B; ++b) s.cu_q[b + 1] = s.cu_q[b] + (c.h_q_lens == nullptr ? 1 : c.h_q_lens[b]);
    }
    if constexpr (kQuantised) {
      if (plan.unpacks) return unpacked_call<N>(heads, s, pools, io, plan, c, r);
    }
    return attend_window<kQuantised, N>(heads, s, pools, io, plan, static_cast<char *>(r.d_workspace), r.stream);
  };
  if (uniform || B <= kFewSeqs) return go(std::integral_constant<int, kFewSeqs>());
  return go(std::integral_constant<int, CPKV_MAX_BATCH>());
}

// Bytes of the workspace of a windowed call.
inline int window_bytes(bool quantised, const HeadArgs &heads, int B, const int32_t *h_q_lens, int64_t max_kv_len, int window, int sinks,
                        int64_t *h_bytes) {
  if (B < 0 || max_kv_len < 0 || window < 0 || sinks < 0 || h_bytes == nullptr) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || max_kv_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  WindowPlan plan;
  rc = window_plan(&plan, heads, quantised, B, h_q_lens, max_kv_len, clamp_window(window, max_kv_len), sinks);
  if (rc != CPKV_OK) return rc;
  *h_bytes = plan.bytes;
  return CPKV_OK;
}

// Bytes of the workspace of a shared call.
inline int shared_bytes(bool quantised, const HeadArgs &heads, int B, int n_groups, const int32_t *h_group_sizes,
                        const int32_t *h_prefix_lens, int64_t max_suffix_len, int64_t *h_bytes) {
  if (B < 0 || n_groups < 0 || max_suffix_len < 0 || h_bytes == nullptr) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || n_groups > CPKV_MAX_BATCH || max_suffix_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  if (n_groups > 0 && (h_group_sizes == nullptr || h_prefix_lens == nullptr)) return CPKV_ERR_ARG;
  SharedPlan plan;
  rc = shared_plan(&plan, heads, quantised, B, n_groups, h_group_sizes, h_prefix_lens, 0, max_suffix_len);
  if (rc != CPKV_OK) return rc;
  *h_bytes = plan.bytes;
  return CPKV_OK;
}

struct SharedCall {
  int B, n_groups;
  const int32_t *h_group_sizes, *h_prefix_lens;
  int64_t max_suffix_len;
  const int32_t *d_prefix_pages;
  int64_t num_prefix_pages;
  const int32_t *d_page_table;
  int64_t table_stride;
  const int32_t *d_suffix_lens;
};

template <bool kQuantised>
int shared_call(const HeadArgs &heads, const RowArgs &rows, const SharedCall &c, const ResultArgs &r) {
  const int B = c.B, n_groups = c.n_groups;
  if (B < 0 || n_groups < 0 || c.max_suffix_len < 0 || (rows.flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || n_groups > CPKV_MAX_BATCH || c.max_suffix_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  PagedPools pools = {};
  rc = open_rows<kQuantised>(&pools, heads, rows);
  if (rc != CPKV_OK) return rc;
  if (n_groups > 0 && (c.h_group_sizes == nullptr || c.h_prefix_lens == nullptr)) return CPKV_ERR_ARG;
  if (c.table_stride < 0 || c.max_suffix_len > c.table_stride * rows.page_size) return CPKV_ERR_CAPACITY;
  SharedPlan plan;
  rc = shared_plan(&plan, heads, kQuantised, B, n_groups, c.h_group_sizes, c.h_prefix_lens, rows.page_size, c.max_suffix_len);
  if (rc != CPKV_OK) return rc;
  if (c.num_prefix_pages < plan.prefix_pages) return CPKV_ERR_CAPACITY;
  if (B == 0) return CPKV_OK;
  if (c.d_suffix_lens == nullptr || r.d_status == nullptr || (c.max_suffix_len > 0 && c.d_page_table == nullptr) ||
      (plan.prefix_pages > 0 && c.d_prefix_pages == nullptr))
    return CPKV_ERR_ARG;
  AttendIo io = {};
  rc = fill_io<kQuantised>(&io, heads, rows, r);
  if (rc != CPKV_OK) return rc;
  if (r.workspace_bytes < plan.bytes) return CPKV_ERR_CAPACITY;
  if (r.d_workspace == nullptr || !aligned16(r.d_workspace)) return CPKV_ERR_ARG;
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    SharedSeqs<N> s = {};
    s.prefix_pages = c.d_prefix_pages;
    s.table = c.d_page_table;
    s.suffix_lens = c.d_suffix_lens;
    s.stride = c.table_stride;
    s.status = r.d_status;
    s.count = n_groups + B;
    s.groups = n_groups;
    s.suffix_cap = (int)c.max_suffix_len;
    int pages = 0;
    for (int g = 0; g < n_groups; ++g) {
      s.cu_q[g + 1] = s.cu_q[g] + c.h_group_sizes[g];
      s.kv[g] = c.h_prefix_lens[g];
      s.page0[g] = pages;
      pages += c.h_prefix_lens[g] / rows.page_size;
    }
    return attend_shared<kQuantised, N>(heads, s, pools, io, plan, static_cast<char *>(r.d_workspace), r.stream);
  };
  if (n_groups <= kFewSeqs) return go(std::integral_constant<int, kFewSeqs>());
  return go(std::integral_constant<int, CPKV_MAX_BATCH>());
}

// The tile kernel over one request, with one head, with waits that run out at once or after `wait_ns`.
template <bool kQuantised>
int selftest_call(const HeadArgs &heads, const RowArgs &rows, int n_tokens, int n_pages, const int32_t *d_page_table,
                  const int32_t *d_kv_len, const ResultArgs &r, int64_t wait_ns) {
  PagedPools pools = {};
  int rc = open_rows<kQuantised>(&pools, heads, rows);
  if (rc != CPKV_OK) return rc;
  AttendIo io = {};
  rc = fill_io<kQuantised>(&io, heads, rows, r);
  if (rc != CPKV_OK) return rc;
  Seqs<kFewSeqs> s = {};
  s.kv_lens = d_kv_len;
  s.table = d_page_table;
  s.stride = n_pages;
  s.status = r.d_status;
  s.count = 1;
  s.kv_cap = n_pages * rows.page_size;
  s.cu_q[1] = n_tokens;
  TileBounds bounds;
  bounds.add(n_tokens, s.kv_cap, 1, 0, 0);  // never finished: one part an item, however long
  TileParams<Seqs<kFewSeqs>> p = {};
  fill_tiles<kQuantised>(&p, s, 1, pools, io, bounds, nullptr, true);
  p.test_wait_ns = (uint64_t)wait_ns;
  return heads.head_dim == 128 ? tile_pass<__nv_bfloat16, 128, kQuantised, true>(p, bounds, r.stream)
                               : tile_pass<__nv_bfloat16, 64, kQuantised, true>(p, bounds, r.stream);
}

}  // namespace
}  // namespace cpkv
