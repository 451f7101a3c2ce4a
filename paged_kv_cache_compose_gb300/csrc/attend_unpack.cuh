// Quantised rows that many query rows attend to, read back into dense pages of the
// element type once: what the tile pass over plain rows then takes.
//
// A tile pass over quantised rows converts a tile of keys for each 256 query rows that
// go over it, and the conversion, not the products, sets its pace (2.0 us a tile, 1.4
// over plain rows).  Reading a key's row back takes 10 kB of traffic at 8 heads of 128, once
// for all query rows (which is the worse of the two for a sequence of few of them in such a call).  Only rows that a query of the sequence sees are read; page p of
// a sequence is dense page first(s) + its place among them, as its table says.
#pragma once

#include "attend.cuh"
#include "quantised.cuh"

namespace cpkv {

constexpr int kDensePage = 32;  // rows of a dense page: the most that a TMA box of the tile pass brings in
constexpr int kUnpackRows = 8;  // rows of a block, one a warp

template <typename S>
struct UnpackParams {
  S seqs;
  PagedPools pools;
  AttendIo io;  // of the quantised rows
  char *rows;   // [page][kDensePage][2][kv_heads][D] of the element type
  int32_t *table;
  int64_t table_stride;
  int cu_pages[S::kArray + 1];  // dense pages before each sequence
};

template <typename T, int D, typename S>
__global__ void __launch_bounds__(kUnpackRows * 32) unpack_kernel(const __grid_constant__ UnpackParams<S> p) {
  const int block = (int)blockIdx.x / (kDensePage / kUnpackRows), part = (int)blockIdx.x % (kDensePage / kUnpackRows);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = upper_index(p.cu_pages, p.seqs.count, block), nq = p.seqs.q_count(s);
  const KeyRange keys = key_range<kDensePage>(p.seqs.kv_len(s), nq, 0, nq, p.seqs.causal, p.seqs.window, p.seqs.sinks);
  const int j = block - p.cu_pages[s];
  if (nq == 0 || j >= keys.n_tiles) return;
  const int start = keys.tile_start(j, kDensePage), key = start + part * kUnpackRows + warp;
  if (part == 0 && threadIdx.x == 0) p.table[s * p.table_stride + start / kDensePage] = block;
  if (!keys.any_sees(key)) return;
  const int page = div_by(key, p.pools.page_size);
  const char *row = page_address(p.pools, p.seqs.pages(s)[page]);
  if (row == nullptr) {
    if (lane == 0) raise_status(p.seqs.status, CPKV_STATUS_PAGE_OOB);
  } else {
    row += (int64_t)(key - page * (int)p.pools.page_size.d) * p.pools.row_bytes;
  }
  const int width = p.io.kv_heads * D;  // elements of the keys, and of the values
  char *const to = p.rows + ((int64_t)block * kDensePage + part * kUnpackRows + warp) * width * 4;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const char *const from = row + (which ? p.io.v_off : p.io.k_off);
    const float *const scales = reinterpret_cast<const float *>(row + (which ? p.io.vs_off : p.io.ks_off));
#pragma unroll 4
    for (int e = lane * 8; e < width; e += 256) {
      const uint2 x = row == nullptr ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2 *>(from + e));
      const float scale = row == nullptr ? 0.f : __ldg(scales + e / D);
      *reinterpret_cast<uint4 *>(to + (int64_t)(which * width + e) * 2) = read_back8<T>(x, scale);
    }
  }
}

}  // namespace cpkv
