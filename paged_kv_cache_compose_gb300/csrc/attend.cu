// Entry points of the attention over paged rows: argument checks, workspace
// layout and the choice of passes.
#include "attend_join.cuh"

namespace cpkv {
namespace {

constexpr int kFewSeqs = 16;

// What both entry points are told of rows, heads and results.
struct HeadArgs {
  int dtype, q_heads, kv_heads, head_dim;
};

int check_heads(const HeadArgs &a) {
  if (a.dtype != CPKV_BF16 && a.dtype != CPKV_FP16) return CPKV_ERR_ARG;
  if (a.kv_heads < 1 || a.q_heads < 1 || a.q_heads % a.kv_heads != 0) return CPKV_ERR_ARG;
  if (a.head_dim != 64 && a.head_dim != 128) return CPKV_ERR_LIMIT;
  if (a.q_heads > 4096 || a.kv_heads > kSplitMaxGrid) return CPKV_ERR_LIMIT;
  return CPKV_OK;
}

int check_rows(const HeadArgs &a, int64_t row_bytes, int64_t k_off, int64_t v_off) {
  const int64_t bytes = (int64_t)a.kv_heads * a.head_dim * 2;
  if (k_off < 0 || v_off < 0 || k_off % 16 != 0 || v_off % 16 != 0) return CPKV_ERR_ARG;
  if (k_off + bytes > row_bytes || v_off + bytes > row_bytes) return CPKV_ERR_ARG;
  return CPKV_OK;
}

int fill_io(AttendIo *io, const HeadArgs &a, const void *q, int64_t q_stride, void *out, int64_t out_stride, float *lse,
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

int64_t round_up(int64_t n, int64_t to) { return ceil_div(n, to) * to; }

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
  // the SMs come to the fewest steps.
  int finish(int kv_heads, int head_dim) {
    const int64_t items = tiles * kv_heads, sms = device_sm_count(), all = steps(max_keys, max_rows);
    int64_t best = INT64_MAX / 16;
    for (int64_t n = 1; n <= std::min<int64_t>(std::max<int64_t>(all / 2, 1), sms) && items > 0; ++n) {
      if (n > 1 && items * n > 4 * sms) break;
      // in 32nds of a step; a part of 256 rows of 128 written and read again is about one
      const int64_t cost = 32 * ceil_div(items * n, sms) * (ceil_div(all, n) + kItemSteps) +
                           (n > 1 ? 32 * kJoinSteps + items * n * head_dim / 128 : 0);
      if (10 * cost < 9 * best) {  // for a tenth or more
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
bool few_rows(int64_t max_rows) { return max_rows <= kSplitRows; }

// How a call is done, from host lengths alone.
struct WindowPlan {
  SplitBounds split;
  TileBounds tile;
  bool few = true, whole = false;
  int64_t tokens = 0, bytes = 0;
};

// A window that no request's keys reach past is none: positions less it stay in 32 bits,
// also below 0 (a request shorter than its queries).
int clamp_window(int window, int64_t max_kv) { return window >= max_kv ? 0 : window; }

int window_plan(WindowPlan *w, const HeadArgs &a, int B, const int32_t *h_q_lens, int64_t max_kv, int window, int sinks) {
  const int group = a.q_heads / a.kv_heads;
  for (int s = 0; s < B; ++s) {
    const int64_t nq = h_q_lens == nullptr ? 1 : h_q_lens[s];
    if (nq < 0) return CPKV_ERR_ARG;
    w->split.add(nq, max_kv, window, sinks);
    w->tile.add(nq, max_kv, group, window, sinks);
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
  const int rc = w->few ? w->split.finish(a.kv_heads) : w->tile.finish(a.kv_heads, a.head_dim);
  w->bytes = w->whole ? 0
             : w->few ? w->split.bytes(B, a.kv_heads, a.head_dim, true)
                      : w->tile.bytes(a.kv_heads, a.head_dim, true);
  return rc;
}

struct SharedPlan {
  SplitBounds split;  // prefixes and suffixes when rows are few
  TileBounds tile;    // and when they are many
  bool few = true;
  int64_t prefix_pages = 0, bytes = 0;
};

int shared_plan(SharedPlan *w, const HeadArgs &a, int B, int n_groups, const int32_t *h_group_sizes,
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
  } else {
    w->tile.add_singles(B, max_suffix);
    rc = w->tile.finish_shared(a.kv_heads);
    w->bytes = w->tile.bytes(a.kv_heads, a.head_dim, false);
  }
  return rc;
}

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
template <typename T, int D, SplitMode kMode, typename S>
int split_pass(SplitParams<S> *p, const SplitBounds &b, cudaStream_t stream) {
  using Shape = SplitShape<D, kMode>;
  const int smem = Shape::kSmem + (kMode == kLine ? (p->seqs.count + 1) * 4 : 0);
  auto kernel = attend_split_kernel<T, D, S, kMode>;
  const int rc = ensure_dynamic_smem((const void *)kernel, Shape::kSmem + (kMode == kLine ? (2 * CPKV_MAX_BATCH + 1) * 4 : 0));
  if (rc != CPKV_OK) return rc;
  int64_t blocks = (int64_t)p->seqs.count * p->io.kv_heads;
  if (kMode == kLine) {  // as many blocks for every head as stay resident together
    const int heads = p->io.kv_heads, resident = persistent_grid((const void *)kernel, kSplitWarps * 32, smem, 8, b.grid_cap);
    blocks = p->space.grid = std::max(resident / heads, 1) * heads;
  }
  if (blocks > INT32_MAX) return CPKV_ERR_LIMIT;
  return launch_kernel(kernel, dim3((unsigned)blocks), dim3(kSplitWarps * 32), smem, false, stream, *p);
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
EncodeTiled encode_tiled() {
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

template <typename S>
void fill_tiles(TileParams<S> *p, const S &seqs, int ragged, const PagedPools &pools, const AttendIo &io,
                const TileBounds &b, char *workspace, bool direct) {
  p->seqs = seqs;
  p->pools = pools;
  p->io = io;
  p->space = b.space(workspace, io.kv_heads);
  p->direct = direct && b.splits == 1;
  p->wide_out = (reinterpret_cast<uintptr_t>(io.out) & 31) == 0 && io.out_stride % 32 == 0;
  fill_maps(p);
  const int group = io.group.d;
  for (int s = 0; s < ragged; ++s)
    p->cu_tiles[s + 1] = p->cu_tiles[s] + (int)ceil_div((int64_t)(seqs.cu_q[s + 1] - seqs.cu_q[s]) * group, kTileRows);
}

template <typename T, int D, bool kTest = false, typename S>
int tile_pass(const TileParams<S> &p, const TileBounds &b, cudaStream_t stream) {
  auto kernel = attend_tile_kernel<T, D, S, kTest>;
  const int rc = ensure_dynamic_smem((const void *)kernel, TileShape<D>::kSmem);
  if (rc != CPKV_OK) return rc;
  const int64_t grid = b.blocks(p.io.kv_heads);
  if (grid > INT32_MAX) return CPKV_ERR_LIMIT;
  return launch_kernel(kernel, dim3((unsigned)grid), dim3(kTileThreads), TileShape<D>::kSmem, false, stream, p);
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

template <int N>
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
        return split_pass<decltype(t), decltype(d)::value, kFewKeys>(&p, plan.split, stream);
      });
    }
    p.space = plan.split.space(workspace, seqs.count, heads.kv_heads, true);
    return for_type_and_dim(heads, [&](auto t, auto d) {
      using T = decltype(t);
      constexpr int D = decltype(d)::value;
      const int rc = split_pass<T, D, kLine>(&p, plan.split, stream);
      return rc != CPKV_OK ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
    });
  }
  TileParams<Seqs<N>> p = {};
  fill_tiles(&p, seqs, seqs.count, pools, io, plan.tile, workspace, true);
  return for_type_and_dim(heads, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    const int rc = tile_pass<T, D>(p, plan.tile, stream);
    return rc != CPKV_OK || p.direct ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
  });
}

// Prefixes and suffixes in one pass, joined.
template <int N>
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
      const int rc = split_pass<T, D, kLine>(&p, plan.split, stream);
      return rc != CPKV_OK ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
    });
  }
  TileParams<SharedSeqs<N>> p = {};
  fill_tiles(&p, seqs, seqs.groups, pools, io, plan.tile, workspace, false);
  return for_type_and_dim(heads, [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    const int rc = tile_pass<T, D>(p, plan.tile, stream);
    return rc != CPKV_OK ? rc : join_pass<T, D>(source_of(p), io, rows, stream);
  });
}

}  // namespace
}  // namespace cpkv

using namespace cpkv;

extern "C" int cpkv_attend_window_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim,
                                                  const int32_t *h_q_lens, int64_t max_kv_len, int window, int sinks,
                                                  int64_t *h_bytes) {
  const HeadArgs heads = {CPKV_BF16, q_heads, kv_heads, head_dim};
  if (B < 0 || max_kv_len < 0 || window < 0 || sinks < 0 || h_bytes == nullptr) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || max_kv_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  window = clamp_window(window, max_kv_len);
  WindowPlan plan;
  rc = window_plan(&plan, heads, B, h_q_lens, max_kv_len, window, sinks);
  if (rc != CPKV_OK) return rc;
  *h_bytes = plan.bytes;
  return CPKV_OK;
}

extern "C" int cpkv_attend_window(int B, int page_size, int cp_size, int dtype, int q_heads, int kv_heads, int head_dim,
                                  int64_t row_bytes, int64_t key_offset, int64_t value_offset,
                                  const int32_t *h_q_lens, int64_t max_kv_len, const void *const *h_pools,
                                  const int64_t *h_pool_cap_pages, const int32_t *d_page_table, int64_t table_stride,
                                  const int32_t *d_kv_lens, int64_t num_tokens, const void *d_q, int64_t q_stride,
                                  float scale, int window, int sinks, void *d_out, int64_t out_stride, float *d_lse, void *d_workspace,
                                  int64_t workspace_bytes, int flags, int32_t *d_status, cpkv_stream_t stream) {
  const HeadArgs heads = {dtype, q_heads, kv_heads, head_dim};
  if (B < 0 || max_kv_len < 0 || window < 0 || sinks < 0 || (flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || max_kv_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  PagedPools pools = {};
  rc = paged_pools(&pools, page_size, cp_size, row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  rc = check_rows(heads, row_bytes, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (table_stride < 0 || max_kv_len > table_stride * page_size) return CPKV_ERR_CAPACITY;
  window = clamp_window(window, max_kv_len);
  WindowPlan plan;
  rc = window_plan(&plan, heads, B, h_q_lens, max_kv_len, window, sinks);
  if (rc != CPKV_OK) return rc;
  if (plan.tokens != num_tokens) return CPKV_ERR_ARG;
  if (plan.tokens == 0) return CPKV_OK;
  if (d_kv_lens == nullptr || d_status == nullptr || (max_kv_len > 0 && d_page_table == nullptr)) return CPKV_ERR_ARG;
  AttendIo io = {};
  rc = fill_io(&io, heads, d_q, q_stride, d_out, out_stride, d_lse, scale, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (workspace_bytes < plan.bytes) return CPKV_ERR_CAPACITY;
  if (plan.bytes > 0 && (d_workspace == nullptr || !aligned16(d_workspace))) return CPKV_ERR_ARG;
  // one query length for all needs no lengths in the kernel's block (the tile kernel goes by them)
  bool uniform = plan.few;
  for (int b = 1; b < B && h_q_lens != nullptr; ++b) uniform &= h_q_lens[b] == h_q_lens[0];
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    Seqs<N> s = {};
    s.kv_lens = d_kv_lens;
    s.table = d_page_table;
    s.stride = table_stride;
    s.status = d_status;
    s.count = B;
    s.kv_cap = (int)max_kv_len;
    s.window = window;
    s.sinks = sinks;
    if (uniform) {
      s.uniform_q = h_q_lens == nullptr ? 1 : h_q_lens[0];
    } else {
      for (int b = 0; b < B; ++b) s.cu_q[b + 1] = s.cu_q[b] + (h_q_lens == nullptr ? 1 : h_q_lens[b]);
    }
    return attend_window<N>(heads, s, pools, io, plan, static_cast<char *>(d_workspace), (cudaStream_t)stream);
  };
  if (uniform || B <= kFewSeqs) return go(std::integral_constant<int, kFewSeqs>());
  return go(std::integral_constant<int, CPKV_MAX_BATCH>());
}

extern "C" int cpkv_attend_shared_workspace_bytes(int B, int n_groups, int q_heads, int kv_heads, int head_dim,
                                                  const int32_t *h_group_sizes, const int32_t *h_prefix_lens,
                                                  int64_t max_suffix_len, int64_t *h_bytes) {
  const HeadArgs heads = {CPKV_BF16, q_heads, kv_heads, head_dim};
  if (B < 0 || n_groups < 0 || max_suffix_len < 0 || h_bytes == nullptr) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || n_groups > CPKV_MAX_BATCH || max_suffix_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  if (n_groups > 0 && (h_group_sizes == nullptr || h_prefix_lens == nullptr)) return CPKV_ERR_ARG;
  SharedPlan plan;
  rc = shared_plan(&plan, heads, B, n_groups, h_group_sizes, h_prefix_lens, 0, max_suffix_len);
  if (rc != CPKV_OK) return rc;
  *h_bytes = plan.bytes;
  return CPKV_OK;
}

extern "C" int cpkv_attend_shared(int B, int n_groups, int page_size, int cp_size, int dtype, int q_heads, int kv_heads,
                                  int head_dim, int64_t row_bytes, int64_t key_offset, int64_t value_offset,
                                  const int32_t *h_group_sizes, const int32_t *h_prefix_lens, int64_t max_suffix_len,
                                  const void *const *h_pools, const int64_t *h_pool_cap_pages,
                                  const int32_t *d_prefix_pages, int64_t num_prefix_pages, const int32_t *d_page_table,
                                  int64_t table_stride, const int32_t *d_suffix_lens, const void *d_q, int64_t q_stride, float scale,
                                  void *d_out, int64_t out_stride, float *d_lse, void *d_workspace,
                                  int64_t workspace_bytes, int flags, int32_t *d_status, cpkv_stream_t stream) {
  const HeadArgs heads = {dtype, q_heads, kv_heads, head_dim};
  if (B < 0 || n_groups < 0 || max_suffix_len < 0 || (flags & ~CPKV_DENSE_PAGES)) return CPKV_ERR_ARG;
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (B > CPKV_MAX_BATCH || n_groups > CPKV_MAX_BATCH || max_suffix_len > INT32_MAX / 2) return CPKV_ERR_LIMIT;
  PagedPools pools = {};
  rc = paged_pools(&pools, page_size, cp_size, row_bytes, h_pools, h_pool_cap_pages, flags);
  if (rc != CPKV_OK) return rc;
  rc = check_rows(heads, row_bytes, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (n_groups > 0 && (h_group_sizes == nullptr || h_prefix_lens == nullptr)) return CPKV_ERR_ARG;
  if (table_stride < 0 || max_suffix_len > table_stride * page_size) return CPKV_ERR_CAPACITY;
  SharedPlan plan;
  rc = shared_plan(&plan, heads, B, n_groups, h_group_sizes, h_prefix_lens, page_size, max_suffix_len);
  if (rc != CPKV_OK) return rc;
  if (num_prefix_pages < plan.prefix_pages) return CPKV_ERR_CAPACITY;
  if (B == 0) return CPKV_OK;
  if (d_suffix_lens == nullptr || d_status == nullptr || (max_suffix_len > 0 && d_page_table == nullptr) ||
      (plan.prefix_pages > 0 && d_prefix_pages == nullptr))
    return CPKV_ERR_ARG;
  AttendIo io = {};
  rc = fill_io(&io, heads, d_q, q_stride, d_out, out_stride, d_lse, scale, key_offset, value_offset);
  if (rc != CPKV_OK) return rc;
  if (workspace_bytes < plan.bytes) return CPKV_ERR_CAPACITY;
  if (d_workspace == nullptr || !aligned16(d_workspace)) return CPKV_ERR_ARG;
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    SharedSeqs<N> s = {};
    s.prefix_pages = d_prefix_pages;
    s.table = d_page_table;
    s.suffix_lens = d_suffix_lens;
    s.stride = table_stride;
    s.status = d_status;
    s.count = n_groups + B;
    s.groups = n_groups;
    s.suffix_cap = (int)max_suffix_len;
    int pages = 0;
    for (int g = 0; g < n_groups; ++g) {
      s.cu_q[g + 1] = s.cu_q[g] + h_group_sizes[g];
      s.kv[g] = h_prefix_lens[g];
      s.page0[g] = pages;
      pages += h_prefix_lens[g] / page_size;
    }
    return attend_shared<N>(heads, s, pools, io, plan, static_cast<char *>(d_workspace), (cudaStream_t)stream);
  };
  if (n_groups <= kFewSeqs) return go(std::integral_constant<int, kFewSeqs>());
  return go(std::integral_constant<int, CPKV_MAX_BATCH>());
}

// The tile kernel over one request with waits that run out at once or after `wait_ns`.
extern "C" int cpkv_selftest_attend_timeout(int head_dim, int n_tokens, int n_pages, const void *d_rows,
                                            const int32_t *d_page_table, const int32_t *d_kv_len, const void *d_q, void *d_out,
                                            int64_t wait_ns, int32_t *d_status, cpkv_stream_t stream) {
  constexpr int kPage = 64;
  const HeadArgs heads = {CPKV_BF16, 1, 1, head_dim};
  int rc = check_heads(heads);
  if (rc != CPKV_OK) return rc;
  if (n_tokens <= kSplitRows || n_pages < 1 || n_pages > (1 << 20) || wait_ns < 0) return CPKV_ERR_ARG;
  if (d_rows == nullptr || d_page_table == nullptr || d_kv_len == nullptr || d_status == nullptr) return CPKV_ERR_ARG;
  const int64_t row_bytes = 4 * head_dim, cap = n_pages;
  PagedPools pools = {};
  rc = paged_pools(&pools, kPage, 1, row_bytes, &d_rows, &cap, CPKV_DENSE_PAGES);
  if (rc != CPKV_OK) return rc;
  AttendIo io = {};
  rc = fill_io(&io, heads, d_q, head_dim, d_out, head_dim, nullptr, 0.125f, 0, 2 * head_dim);
  if (rc != CPKV_OK) return rc;
  Seqs<kFewSeqs> s = {};
  s.kv_lens = d_kv_len;
  s.table = d_page_table;
  s.stride = n_pages;
  s.status = d_status;
  s.count = 1;
  s.kv_cap = n_pages * kPage;
  s.cu_q[1] = n_tokens;
  TileBounds bounds;
  bounds.add(n_tokens, s.kv_cap, 1, 0, 0);  // never finished: one part an item, however long
  TileParams<Seqs<kFewSeqs>> p = {};
  fill_tiles(&p, s, 1, pools, io, bounds, nullptr, true);
  p.test_wait_ns = (uint64_t)wait_ns;
  return head_dim == 128 ? tile_pass<__nv_bfloat16, 128, true>(p, bounds, (cudaStream_t)stream)
                         : tile_pass<__nv_bfloat16, 64, true>(p, bounds, (cudaStream_t)stream);
}
