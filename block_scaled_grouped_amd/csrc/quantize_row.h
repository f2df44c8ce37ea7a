// Rows in 8-bit integers with a float32 scale each:
//
//   s = float32(max_i |x_i| / 127),   q_i = the integer nearest to x_i / s, ties to even
//
// of the exact quotient.  A product by the reciprocal of s is off by a few steps of 2^-24,
// so the integer that it rounds to can be the wrong one only next to a border; the rest
// x - q s is exact in float32 (x has 8 or 11 bits and s 24, so that the rest's bits lie
// between the last of s and half of s), and where it reaches s / 2 the integer is moved.
// |q| <= 127: |x| / s is at most 127 (1 + 2^-24), or 127.13 where s is so small that it
// has only 9 bits.  A row of zeros has s = 0 and q = 0; one with an infinity or a NaN has
// s = NaN and q = 0.
#ifndef BSG_QUANTIZE_ROW_H
#define BSG_QUANTIZE_ROW_H

#include "bsg_internal.h"

namespace bsg {
namespace {

template <bool F16>
__device__ __forceinline__ float elem(uint32_t word, int h) {
  const uint32_t bits = h ? word >> 16 : word & 0xffffu;
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  return h ? __uint_as_float(word & 0xffff0000u) : __uint_as_float(word << 16);
}

// Largest magnitude bits of the halves of a and b, half by half.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));
  const v2u16 x = __builtin_bit_cast(v2u16, a & 0x7fff7fffu);
  const v2u16 y = __builtin_bit_cast(v2u16, b & 0x7fff7fffu);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}

// m and the 8 values of v.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, const v4i& v) {
  return max2(m, max2(max2((uint32_t)v[0], (uint32_t)v[1]), max2((uint32_t)v[2], (uint32_t)v[3])));
}

struct RowScale {
  float s;        // as it is stored
  float up;       // power of two that takes the row to normal numbers
  float su, inv;  // s * up and its reciprocal
  float half;     // s * up / 2
};

// bits: the row's largest magnitude, as its 16 bits.
template <bool F16>
__device__ __forceinline__ RowScale row_scale(uint32_t bits, bool& finite) {
  finite = bits < (F16 ? 0x7c00u : 0x7f80u);
  const float amax = elem<F16>(bits, 0);
  RowScale r;
  r.s = amax / 127.0f;
  r.up = r.s < 0x1p-60f ? 0x1p80f : 1.0f;
  r.su = r.s * r.up;
  r.inv = finite && r.s > 0.0f ? 1.0f / r.su : 0.0f;
  r.half = 0.5f * r.su;
  if (!finite) {
    r.s = __uint_as_float(0x7fc00000u);
    r.su = 0.0f;
    r.half = __uint_as_float(0x7f800000u);
  }
  return r;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

// The integers of 8 elements, as bytes.
template <bool F16>
__device__ __forceinline__ v2i quantize8(const v4i& v, const RowScale& r, bool finite) {
  float t[8], rest[8];
  bool border = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = elem<F16>((uint32_t)v[e >> 1], e & 1) * r.up;
    t[e] = fmaf(x, r.inv, kMagic);
    rest[e] = fmaf(kMagic - t[e], r.su, x);
    border |= fabsf(rest[e]) >= r.half;
  }
  if (__any(border) && finite && r.inv != 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool odd = (__float_as_uint(t[e]) & 1u) != 0;
      const float a = fabsf(rest[e]);
      if (a > r.half || (a == r.half && odd)) t[e] += rest[e] > 0.0f ? 1.0f : -1.0f;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // the low byte of each sum is the integer
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 1]),
                                              __float_as_uint(t[4 * h]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(t[4 * h + 3]),
                                              __float_as_uint(t[4 * h + 2]), 0x04000c0cu);
    w[h] = finite ? lo | hi : 0u;
  }
  return v2i{(int)w[0], (int)w[1]};
}

}  // namespace
}  // namespace bsg

#endif  // BSG_QUANTIZE_ROW_H
