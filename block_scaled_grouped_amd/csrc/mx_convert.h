// Conversions of 16-bit values to MXFP8 codes and their block scales, shared by the
// kernels that write them.
#ifndef BSG_MX_CONVERT_H
#define BSG_MX_CONVERT_H

#include "bsg_internal.h"

namespace bsg {
namespace {

// E8M0 byte from the largest bf16 magnitude bits of a block: the OCP rule,
// exponent(amax) - emax of the element format (8 for E4M3, 15 for E5M2).
template <bool E5M2 = false>
__device__ __forceinline__ uint32_t e8m0_from_amax_bits(uint32_t amax_bits) {
  constexpr uint32_t emax = E5M2 ? 15u : 8u;
  const uint32_t e = amax_bits >> 7;  // biased exponent of the bf16 magnitude
  return e > emax ? e - emax : 0u;
}

// The scale operand of the scaled converts: a float whose exponent field is the
// E8M0 byte (the instruction reads only the exponent field).
__device__ __forceinline__ float e8m0_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

typedef unsigned short v2u16 __attribute__((ext_vector_type(2)));

// Lane moves inside 16-lane rows (DPP): the value of lane l ^ 1, and of lane
// l + N (only read where l + N stays inside the row).
__device__ __forceinline__ uint32_t dpp_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);  // quad_perm 1,0,3,2
}
template <int N>
__device__ __forceinline__ uint32_t dpp_down(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x100 + N, 0xF, 0xF, false);  // row_shl N
}

// Largest of the two bf16 magnitudes in each 16-bit half of a and b.
__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b) {
  const v2u16 x = __builtin_bit_cast(v2u16, a & 0x7fff7fffu);
  const v2u16 y = __builtin_bit_cast(v2u16, b & 0x7fff7fffu);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
}

// Combines the two halves of an amax2 result.
__device__ __forceinline__ uint32_t amax_fold(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// Overflowed codes become the largest finite code, in each byte of a word:
// E4M3 S.1111.111 (only produced for magnitudes above 464) -> S.1111.110;
// E5M2 S.11111.00 (the infinity the E5M2 convert gives past 57344, the only
// exponent-31 code finite input produces) -> S.11110.11.
template <bool E5M2 = false>
__device__ __forceinline__ uint32_t fp8_saturate(uint32_t x) {
  constexpr uint32_t gap = E5M2 ? 0x04040404u : 0x01010101u;  // 0x80 - first overflow code
  const uint32_t t = (((x & 0x7f7f7f7fu) + gap) >> 7) & 0x01010101u;
  // E4M3: S.1111.111 -> S.1111.110 flips bit 0 (one bitwise op with the mask)
  return E5M2 ? x - t : x ^ t;
}

// Two packed bf16 (low element first), scaled -> two E4M3 (or E5M2) bytes in
// the low (HI = false) or high half of `old`.  Both converts are exact
// round-to-nearest-even of x / 2^scale up to the overflow handled above.
template <bool HI, bool E5M2 = false>
__device__ __forceinline__ uint32_t cvt2(uint32_t w, float scale, uint32_t old) {
  v2s r;
  if constexpr (E5M2)
    r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(__builtin_bit_cast(v2s, old),
                                                  __builtin_bit_cast(v2bf, w), scale, HI);
  else
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(__builtin_bit_cast(v2s, old),
                                                  __builtin_bit_cast(v2bf, w), scale, HI);
  return __builtin_bit_cast(uint32_t, r);
}

// 8 bf16 (4 dwords) -> 8 E4M3 (or E5M2) bytes (2 dwords).
template <bool E5M2 = false>
__device__ __forceinline__ uint2 cvt8(uint4 v, float scale) {
  // The first convert's other half is written by the second, so its prior
  // contents do not matter: passing the source word lets the result take the
  // source's register (no copy into a zeroed one).
  const uint32_t lo = cvt2<true, E5M2>(v.y, scale, cvt2<false, E5M2>(v.x, scale, v.x));
  const uint32_t hi = cvt2<true, E5M2>(v.w, scale, cvt2<false, E5M2>(v.z, scale, v.z));
  return make_uint2(fp8_saturate<E5M2>(lo), fp8_saturate<E5M2>(hi));
}

}  // namespace
}  // namespace bsg

#endif  // BSG_MX_CONVERT_H
