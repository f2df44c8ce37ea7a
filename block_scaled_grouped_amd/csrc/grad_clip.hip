// Global norm of many gradient tensors, and their clipping by it.
//
//   norm = sqrt(sum over all tensors of x^2)
//   y    = x * min(1, max_norm / (norm + 1e-6))
//
// The tensors are cut on the host into chunks (a plan, made once for buffers
// that stay where they are); a launch walks the chunks whatever tensors they
// belong to, so the number of tensors costs no launches.
//
// Squares and sums are held in 64 bits: a square of a 32-bit value neither
// overflows nor vanishes there, and the order of the sums is fixed (thread,
// block, then the blocks' sums in one order), so a norm repeats bit for bit.
// The multiply-adds are far from the vector units' 64-bit rate.
#include "bsg_internal.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;

// Addresses come from the plan, so the compiler has to be told that they are global.
// 16 bytes at p are aligned to their elements only.
typedef __attribute__((address_space(1))) char gchar;
typedef v4i v4i_any __attribute__((aligned(2)));
typedef __attribute__((address_space(1))) v4i_any gv4i;
__device__ __forceinline__ v4i load16(const gchar* p) {
  return *reinterpret_cast<const gv4i*>(p);
}
// The scaling pass goes by what the caches still hold of the first pass, so what it
// has read and what it writes are not kept there (300 bf16 tensors of 200 M elements:
// 241 -> 200 us).
__device__ __forceinline__ v4i load16_last(const gchar* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(p));
}
__device__ __forceinline__ void store16_last(gchar* p, const v4i& v) {
  __builtin_nontemporal_store(v, reinterpret_cast<gv4i*>(p));
}

// dtype 0: bf16, 1: fp16, 2: float32.
template <int DT>
__device__ __forceinline__ float elem(const v4i& v, int e) {
  if constexpr (DT == 2) return __int_as_float(v[e]);
  const uint32_t bits = ((uint32_t)v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
  return bf16_to_f32(bits);
}

// The element at index i, alone.
template <int DT>
__device__ __forceinline__ float one_elem(const gchar* src, int i) {
  if constexpr (DT == 2)
    return *reinterpret_cast<const __attribute__((address_space(1))) float*>(src + (int64_t)i * 4);
  const uint16_t b =
      *reinterpret_cast<const __attribute__((address_space(1))) uint16_t*>(src + (int64_t)i * 2);
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, b);
  return bf16_to_f32(b);
}

// Pieces of 16 bytes that a thread has in flight.
constexpr int kFlight = 4;

template <int DT>
__device__ __forceinline__ double chunk_sumsq(const GradChunk& c) {
  constexpr int per = DT == 2 ? 4 : 8;
  const gchar* src = (const gchar*)c.src;
  const int whole = c.n / per;
  double s = 0.0;
  int i = threadIdx.x;
  for (; i + (kFlight - 1) * kThreads < whole; i += kFlight * kThreads) {
    v4i v[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) v[f] = load16(src + (int64_t)(i + f * kThreads) * 16);
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
#pragma unroll
      for (int e = 0; e < per; ++e) {
        const double x = (double)elem<DT>(v[f], e);
        s += x * x;
      }
  }
  for (; i < whole; i += kThreads) {
    const v4i v = load16(src + (int64_t)i * 16);
#pragma unroll
    for (int e = 0; e < per; ++e) {
      const double x = (double)elem<DT>(v, e);
      s += x * x;
    }
  }
  const int tail = whole * per + threadIdx.x;
  if (tail < c.n) {
    const double x = (double)one_elem<DT>(src, tail);
    s += x * x;
  }
  return s;
}

__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads / 64];
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) t += part[i];
  return t;
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const GradChunk* __restrict__ plan,
                                                              int64_t num_chunks,
                                                              double* __restrict__ partials) {
  double s = 0.0;
  for (int64_t i = blockIdx.x; i < num_chunks; i += gridDim.x) {
    const GradChunk c = plan[i];
    if (c.dtype == 2) s += chunk_sumsq<2>(c);
    else if (c.dtype == 1) s += chunk_sumsq<1>(c);
    else s += chunk_sumsq<0>(c);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__device__ __forceinline__ double sum_partials(const double* __restrict__ partials, int count) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) s += partials[i];
  return block_sum(s);
}

__device__ __forceinline__ void write_norm(double sumsq, float* norm, double* out_sumsq,
                                           uint32_t* status) {
  const float n = (float)sqrt(sumsq);
  if (norm != nullptr) *norm = n;
  if (out_sumsq != nullptr) *out_sumsq = sumsq;
  // the norm as the caller gets it: a finite sum's may be past float32's largest value
  if (!(n < __builtin_inff())) dev_status_or(status, kDevNonFinite);
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* __restrict__ partials,
                                                             int count, float* norm,
                                                             double* out_sumsq, uint32_t* status) {
  const double s = sum_partials(partials, count);
  if (threadIdx.x == 0) write_norm(s, norm, out_sumsq, status);
}

// A factor in two steps, x * a * b.  A norm of more than max_norm * 2^126 makes factors below
// float32's normal numbers, where fewer than 24 bits are left of them: there a is the factor
// times 2^64 and b 2^-64.  Elsewhere b is 1, which changes nothing.
struct Factor {
  float a, b;
};
__device__ __forceinline__ Factor make_factor(double f) {
  if (f < 0x1p-126) return {(float)(f * 0x1p64), 0x1p-64f};
  return {(float)f, 1.0f};
}
__device__ __forceinline__ float times(float x, const Factor& f) { return x * f.a * f.b; }

template <int DT>
__device__ __forceinline__ v4i scaled(const v4i& v, const Factor& f) {
  v4i y;
  if constexpr (DT == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __float_as_int(times(elem<2>(v, e), f));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[e] = (int)pack16<DT == 1>(times(elem<DT>(v, 2 * e), f), times(elem<DT>(v, 2 * e + 1), f));
  }
  return y;
}

template <int DT>
__device__ __forceinline__ void chunk_scale(const GradChunk& c, const Factor& f) {
  constexpr int per = DT == 2 ? 4 : 8;
  const gchar* src = (const gchar*)c.src;
  gchar* dst = (gchar*)c.dst;
  const int whole = c.n / per;
  int i = threadIdx.x;
  for (; i + (kFlight - 1) * kThreads < whole; i += kFlight * kThreads) {
    v4i v[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) v[q] = load16_last(src + (int64_t)(i + q * kThreads) * 16);
#pragma unroll
    for (int q = 0; q < kFlight; ++q)
      store16_last(dst + (int64_t)(i + q * kThreads) * 16, scaled<DT>(v[q], f));
  }
  for (; i < whole; i += kThreads)
    store16_last(dst + (int64_t)i * 16, scaled<DT>(load16_last(src + (int64_t)i * 16), f));
  const int tail = whole * per + threadIdx.x;
  if (tail < c.n) {
    const float x = times(one_elem<DT>(src, tail), f);
    if constexpr (DT == 2) {
      *reinterpret_cast<__attribute__((address_space(1))) float*>(dst + (int64_t)tail * 4) = x;
    } else {
      *reinterpret_cast<__attribute__((address_space(1))) uint16_t*>(dst + (int64_t)tail * 2) =
          (uint16_t)(pack16<DT == 1>(x, x) & 0xffffu);
    }
  }
}

// Every block adds the partial sums again, in the same order (2048 of them at
// most, from the L2): cheaper than a third launch between the two passes.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(
    const GradChunk* __restrict__ plan, int64_t num_chunks, const double* __restrict__ partials,
    int count, float max_norm, float* norm, uint32_t* status) {
  const double sumsq = sum_partials(partials, count);
  if (blockIdx.x == 0 && threadIdx.x == 0) write_norm(sumsq, norm, nullptr, status);
  double f = (double)max_norm / (sqrt(sumsq) + 1e-6);
  if (f > 1.0) f = 1.0;  // a NaN stays one
  const Factor factor = make_factor(f);
  // the second pass begins with what the first one read last
  for (int64_t i = num_chunks - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const GradChunk c = plan[i];
    if (factor.a == 1.0f && factor.b == 1.0f && c.dst == c.src) continue;
    if (c.dtype == 2) chunk_scale<2>(c, factor);
    else if (c.dtype == 1) chunk_scale<1>(c, factor);
    else chunk_scale<0>(c, factor);
  }
}

int blocks_for(int64_t num_chunks) {
  int64_t b = 8 * (int64_t)device_cu_count();
  if (b > kGradMaxBlocks) b = kGradMaxBlocks;
  if (b > num_chunks) b = num_chunks;
  return (int)(b > 0 ? b : 1);
}

}  // namespace

hipError_t launch_grad_norm(const GradChunk* plan, int64_t num_chunks, double* partials,
                            float* norm, double* sumsq, uint32_t* status, hipStream_t stream) {
  const int blocks = blocks_for(num_chunks);
  hipLaunchKernelGGL(grad_sumsq_kernel, dim3(blocks), dim3(kThreads), 0, stream, plan, num_chunks,
                     partials);
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, partials, blocks, norm,
                     sumsq, status);
  return hipGetLastError();
}

hipError_t launch_clip_grad_norm(const GradChunk* plan, int64_t num_chunks, float max_norm,
                                 const double* sumsq, double* partials, float* norm,
                                 uint32_t* status, hipStream_t stream) {
  const int blocks = blocks_for(num_chunks);
  if (sumsq == nullptr)
    hipLaunchKernelGGL(grad_sumsq_kernel, dim3(blocks), dim3(kThreads), 0, stream, plan, num_chunks,
                       partials);
  hipLaunchKernelGGL(grad_scale_kernel, dim3(blocks), dim3(kThreads), 0, stream, plan, num_chunks,
                     sumsq != nullptr ? sumsq : partials, sumsq != nullptr ? 1 : blocks, max_norm,
                     norm, status);
  return hipGetLastError();
}

}  // namespace bsg
