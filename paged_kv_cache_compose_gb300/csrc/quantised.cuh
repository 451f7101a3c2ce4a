// Quantised rows: e4m3 values with float scales.
//
// A group of elements (a key head of 64 or 128, 128 values or a value head of 64)
// shares a scale s, the smallest power of two (2^-126 at least) whose 448-fold
// reaches the largest magnitude of its finite elements; an element x is kept as
// e4m3(x / s), rounded once to nearest even, an infinity or a NaN as e4m3's NaN.
// A power of two loses none of the three bits of fraction (448 is the largest e4m3
// number: the largest element falls into (224, 448]), makes the division exact, and
// the product s * e4m3 of a row read back exact in bf16 within that type's range (multiples of
// 2^-133, less than 2^128).  Readers take any scale.
#pragma once

#include "paged.cuh"

namespace cpkv {

constexpr int kValueGroup = 128;  // values of a scale (64 where that is a whole head)

inline int value_group(const cpkv_quantised_row &r) { return r.value_dim < kValueGroup ? r.value_dim : kValueGroup; }

// Bytes of a row's key, value, key scale and value scale parts.
struct RowParts {
  int64_t at[4], bytes[4];
};

inline RowParts row_parts(const cpkv_quantised_row &r) {
  const int64_t heads = r.kv_heads;
  return RowParts{{r.key_offset, r.value_offset, r.key_scale_offset, r.value_scale_offset},
                  {heads * r.key_dim * (r.keep_keys ? 2 : 1), heads * r.value_dim, r.keep_keys ? 0 : heads * 4,
                   heads * (r.value_dim / value_group(r)) * 4}};
}

// Whether rows can be kept so: widths, alignment, parts inside the row and apart.
inline int check_quantised_row(const cpkv_quantised_row *r) {
  if (r == nullptr || r->kv_heads < 1 || r->key_dim <= 0 || r->value_dim <= 0) return CPKV_ERR_ARG;
  if (r->kv_heads > 1024 || r->key_dim > 4096 || r->value_dim > 4096) return CPKV_ERR_LIMIT;
  if (r->keep_keys ? r->key_dim % 8 != 0 || r->key_dim > 512 : r->key_dim != 64 && r->key_dim != 128) return CPKV_ERR_LIMIT;
  if (r->value_dim != 64 && r->value_dim % kValueGroup != 0) return CPKV_ERR_LIMIT;
  const RowParts parts = row_parts(*r);
  for (int i = 0; i < 4; ++i) {
    if (parts.bytes[i] == 0) continue;
    if (parts.at[i] < 0 || parts.at[i] % (i < 2 ? 16 : 4) != 0 || parts.at[i] > r->row_bytes - parts.bytes[i]) return CPKV_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (parts.bytes[j] > 0 && parts.at[i] < parts.at[j] + parts.bytes[j] && parts.at[j] < parts.at[i] + parts.bytes[i])
        return CPKV_ERR_ARG;
  }
  return CPKV_OK;
}

// x, or NaN where it is infinite.
CPKV_DEV float finite_or_nan(float x) { return x + (x - x); }

// The group's scale from its largest magnitude, and the factor that divides by it:
// 448 = 1.75 * 2^8, so the exponent is that of the magnitude less 8, and one more
// where the fraction is past .75.
struct GroupScale {
  float scale, inverse;
};

CPKV_DEV GroupScale group_scale(float largest) {
  const int e = max((int)((__float_as_uint(largest) + 0x1fffffu) >> 23) - 8, 1);
  return GroupScale{__uint_as_float((uint32_t)e << 23), __uint_as_float((uint32_t)(254 - e) << 23)};
}

// The exponent of the scale, -126 to 127, from the largest magnitude in 64 bits; and the most
// that a scale reaches, 448 * 2^127: what is larger is kept as an infinity is.
CPKV_DEV int group_exponent(double largest) {
  return max((int)((__double_as_longlong(largest) + 0x3ffffffffffffll) >> 52) - 8 - 1023, -126);
}
constexpr double kMostQuantised = 0x1.cp135;

// Four numbers rounded to e4m3, the first in the lowest byte.
CPKV_DEV uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)hi << 16 | lo;
}

// The two e4m3 numbers of the low (high) half as a pair of fp16, which holds every one of them.
CPKV_DEV uint32_t halves_low(uint32_t v) {
  uint32_t r;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(v));
  return r;
}
CPKV_DEV uint32_t halves_high(uint32_t v) {
  uint32_t r;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\ncvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(v));
  return r;
}

// Two e4m3 numbers (as halves) times a scale, in the element type; a number past
// fp16's largest becomes the largest (448 times the scale of 65504's group is more).
template <typename T>
CPKV_DEV uint32_t read_back2(uint32_t halves, float scale) {
  const float2 x = unpack2<__half>(halves);
  float a, b;
  asm("{\n.reg .b64 x, s;\nmov.b64 x, {%2, %3};\nmov.b64 s, {%4, %4};\nmul.rn.f32x2 x, x, s;\nmov.b64 {%0, %1}, x;\n}"
      : "=f"(a), "=f"(b)
      : "f"(x.x), "f"(x.y), "f"(scale));
  if constexpr (std::is_same<T, __half>::value) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  return pack2<T>(a, b);
}

// Eight e4m3 numbers times a scale.
template <typename T>
CPKV_DEV uint4 read_back8(uint2 v, float scale) {
  return make_uint4(read_back2<T>(halves_low(v.x), scale), read_back2<T>(halves_high(v.x), scale),
                    read_back2<T>(halves_low(v.y), scale), read_back2<T>(halves_high(v.y), scale));
}

}  // namespace cpkv
