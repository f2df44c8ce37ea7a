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
//
// HBM bound: 2 bytes in and 1 out an element.  A row stays in registers between its
// maximum and its integers.
#include "bsg_internal.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;

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

struct Args {
  const uint16_t* x;
  int64_t ldx, rows_cap, cols;
  const int64_t* offsets;  // or null: all rows
  int G;
  int8_t* data;
  float* scales;
  uint32_t* status;
};

// TPR threads take a row, NC runs of 8 elements each: a row of at most 8 TPR NC elements
// is read once (LONG: any length, read again from the caches for its integers).
template <bool F16, int TPR, int NC, bool LONG>
__global__ __launch_bounds__(kThreads) void quantize_int8_kernel(Args p) {
  constexpr int kRows = kThreads / TPR;
  __shared__ uint32_t peak[kThreads / 64];
  int64_t first = 0, last = p.rows_cap;
  if (p.offsets != nullptr) {
    first = p.offsets[0];
    last = p.offsets[p.G];
    const uint32_t bad = (first < 0 || last < first ? kDevNegativeSize : 0u) |
                         (last > p.rows_cap ? kDevOverCapacity : 0u);
    if (bad != 0 && blockIdx.x == 0 && threadIdx.x == 0) dev_status_or(p.status, bad);
    if (first < 0) first = 0;
    if (last > p.rows_cap) last = p.rows_cap;
  }
  const int t = threadIdx.x % TPR;
  const int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  if (row >= last) return;  // of a whole wave, and where rows share barriers of the workgroup
  const uint16_t* src = p.x + row * p.ldx;
  const int cols = (int)p.cols;
  v4i v[NC];
  uint32_t m = 0;
  for (int base = 0; base < (LONG ? cols : 1); base += 8 * TPR * NC) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = base + 8 * (t + TPR * c);
      v[c] = v4i{0, 0, 0, 0};
      if (e < cols) {
        const v4i* at = reinterpret_cast<const v4i*>(src + e);
        v[c] = LONG ? *at : __builtin_nontemporal_load(at);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
      m = max2(m, max2(max2((uint32_t)v[c][0], (uint32_t)v[c][1]),
                       max2((uint32_t)v[c][2], (uint32_t)v[c][3])));
  }
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) peak[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) m = max(m, peak[w]);
  }
  bool finite;
  const RowScale r = row_scale<F16>(m, finite);
  if (t == 0) {
    p.scales[row] = r.s;
    if (!finite) dev_status_or(p.status, kDevNonFinite);
  }
  int8_t* dst = p.data + row * p.cols;
  for (int base = 0; base < (LONG ? cols : 1); base += 8 * TPR * NC) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = base + 8 * (t + TPR * c);
      if constexpr (LONG) {
        if (e < cols) v[c] = *reinterpret_cast<const v4i*>(src + e);
      }
      const v2i q = quantize8<F16>(v[c], r, finite);
      if (e < cols) *reinterpret_cast<v2i*>(dst + e) = q;
    }
  }
}

template <bool F16, int TPR, int NC, bool LONG>
hipError_t launch(const Args& p, hipStream_t stream) {
  constexpr int kRows = kThreads / TPR;
  const int64_t blocks = (p.rows_cap + kRows - 1) / kRows;
  hipLaunchKernelGGL((quantize_int8_kernel<F16, TPR, NC, LONG>), dim3((unsigned)blocks),
                     dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_type(const Args& p, hipStream_t stream) {
  if (p.cols <= 512) return launch<F16, 64, 1, false>(p, stream);
  if (p.cols <= 1024) return launch<F16, 64, 2, false>(p, stream);
  if (p.cols <= 2048) return launch<F16, 64, 4, false>(p, stream);
  if (p.cols <= 4096) return launch<F16, 256, 2, false>(p, stream);
  if (p.cols <= 8192) return launch<F16, 256, 4, false>(p, stream);
  if (p.cols <= 16384) return launch<F16, 256, 8, false>(p, stream);
  return launch<F16, 256, 4, true>(p, stream);
}

}  // namespace

hipError_t launch_quantize_int8(int f16, const void* x, int64_t ldx, int64_t rows_cap, int64_t cols,
                                int G, const int64_t* offsets, int8_t* data, float* scales,
                                uint32_t* status, hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const Args p{static_cast<const uint16_t*>(x), ldx, rows_cap, cols, offsets, G, data, scales,
               status};
  return f16 ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

}  // namespace bsg
