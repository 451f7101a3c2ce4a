// Paged token rows as the serving operators address them: owner pools of
// pages of page_size rows, 16-bit element types, and division by run-time
// constants.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace cpkv {

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994): with
// s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// floor(n / d) = (mulhi(n, m) + n) >> s.
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.s = 0;
  while ((1ull << f.s) < d) ++f.s;
  f.m = (uint32_t)(((1ull << 32) * ((1ull << f.s) - d)) / d + 1);
  return f;
}

CPKV_DEV int div_by(int n, const FastDiv &f) { return (int)((__umulhi((uint32_t)n, f.m) + (uint32_t)n) >> f.s); }

// The owner pools of one paged cache.  Logical page lp is page lp / cp of
// pool lp % cp; ids below first_page or beyond a pool's capacity are invalid.
struct PagedPools {
  char *pool[CPKV_MAX_CP];
  int32_t cap[CPKV_MAX_CP];
  int64_t row_bytes, page_bytes;
  FastDiv page_size, cp;
  int first_page;
};

// Address of a page, null when the id is invalid.
CPKV_DEV char *page_address(const PagedPools &p, int page) {
  if (page < p.first_page) return nullptr;
  const int local = div_by(page, p.cp);
  const int owner = page - local * (int)p.cp.d;
  if (local >= p.cap[owner]) return nullptr;
  return p.pool[owner] + (int64_t)local * p.page_bytes;
}

// Fills the pools from an entry point's arguments; the return code of a bad
// one (null or unaligned pool, capacity below zero, sizes off 16 bytes).
inline int paged_pools(PagedPools *p, int page_size, int cp_size, int64_t row_bytes, const void *const *h_pools,
                       const int64_t *h_cap, int flags) {
  if (page_size <= 0 || cp_size < 1 || row_bytes <= 0 || row_bytes % 16 != 0) return CPKV_ERR_ARG;
  if (cp_size > CPKV_MAX_CP || row_bytes > INT32_MAX) return CPKV_ERR_LIMIT;
  if (h_pools == nullptr || h_cap == nullptr) return CPKV_ERR_ARG;
  for (int r = 0; r < cp_size; ++r) {
    if (h_cap[r] < 0 || (h_cap[r] > 0 && h_pools[r] == nullptr) || !aligned16(h_pools[r])) return CPKV_ERR_ARG;
    p->pool[r] = static_cast<char *>(const_cast<void *>(h_pools[r]));
    p->cap[r] = (int32_t)std::min<int64_t>(h_cap[r], INT32_MAX);
  }
  p->row_bytes = row_bytes;
  p->page_bytes = row_bytes * page_size;
  p->page_size = fast_div((uint32_t)page_size);
  p->cp = fast_div((uint32_t)cp_size);
  p->first_page = (flags & CPKV_DENSE_PAGES) ? 0 : 1;
  return CPKV_OK;
}

// ---------------------------------------------------------------------------
// 16-bit element types
// ---------------------------------------------------------------------------
template <typename T>
CPKV_DEV float2 unpack2(uint32_t v);
template <>
CPKV_DEV float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
CPKV_DEV float2 unpack2<__half>(uint32_t v) {
  __half2 h;
  memcpy(&h, &v, 4);
  return __half22float2(h);
}

// Two floats rounded to nearest even, `lo` in the low half.
template <typename T>
CPKV_DEV uint32_t pack2(float lo, float hi);
template <>
CPKV_DEV uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
CPKV_DEV uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// acc + 0 v in both halves: from an acc of 0, 0 unless v holds an infinity or a NaN.
template <typename T>
CPKV_DEV uint32_t mark_infinite(uint32_t v, uint32_t acc);
template <>
CPKV_DEV uint32_t mark_infinite<__nv_bfloat16>(uint32_t v, uint32_t acc) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0), "r"(acc));
  return r;
}
template <>
CPKV_DEV uint32_t mark_infinite<__half>(uint32_t v, uint32_t acc) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0), "r"(acc));
  return r;
}
template <typename T>
CPKV_DEV uint4 mark_infinite(const uint4 &v, const uint4 &acc) {
  return make_uint4(mark_infinite<T>(v.x, acc.x), mark_infinite<T>(v.y, acc.y), mark_infinite<T>(v.z, acc.z),
                    mark_infinite<T>(v.w, acc.w));
}

// The infinities and NaNs of a pair, zeros for the other numbers; and the reverse.
template <typename T>
CPKV_DEV uint32_t infinite_of(uint32_t v) {
  constexpr uint32_t kExponent = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return ((v & kExponent) == kExponent ? v & 0xffffu : 0u) | (((v >> 16) & kExponent) == kExponent ? v & 0xffff0000u : 0u);
}
template <typename T>
CPKV_DEV uint32_t finite_of(uint32_t v) {
  return v ^ infinite_of<T>(v);
}

}  // namespace cpkv
