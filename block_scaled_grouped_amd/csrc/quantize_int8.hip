// Rows in 8-bit integers with a float32 scale each (quantize_row.h has the mathematics).
//
// HBM bound: 2 bytes in and 1 out an element.  A row stays in registers between its
// maximum and its integers.
#include "bsg_internal.h"
#include "quantize_row.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;

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
// is read once (LONG: any length, read again from the caches for its integers).  STREAM: the
// integers go past the caches.
template <bool F16, int TPR, int NC, bool LONG, bool STREAM>
__global__ __launch_bounds__(kThreads) void quantize_int8_kernel(Args p) {
  constexpr int kRows = kThreads / TPR;
  __shared__ uint32_t peak[2][kThreads / 64];
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
  const int cols = (int)p.cols;
  int turn = 0;
  for (int64_t row = first + (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < last;
       row += (int64_t)gridDim.x * kRows) {  // the same for all threads that share a barrier
    const uint16_t* src = p.x + row * p.ldx;
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
      for (int c = 0; c < NC; ++c) m = max_magnitude(m, v[c]);
    }
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    if constexpr (TPR > 64) {
      if ((threadIdx.x & 63) == 0) peak[turn][threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) m = max(m, peak[turn][w]);
      turn ^= 1;  // the next row's go elsewhere: one barrier a row
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
        if (e < cols) {
          v2i* at = reinterpret_cast<v2i*>(dst + e);
          if constexpr (STREAM) __builtin_nontemporal_store(q, at);
          else *at = q;
        }
      }
    }
  }
}

// Integers of so many bytes go past the caches: 114688 x 4096 (470 MB) 224 us without and 216 with
// it (6.5 TB/s), the tokens and the product of 32768 x 7168 (242 MB) 560 and 556, of 16384 x 4096
// (67 MB) 795 both.  Fewer stay there for the product that reads them.
constexpr int64_t kStreamBytes = (int64_t)96 << 20;

template <bool F16, int TPR, int NC, bool LONG>
hipError_t launch(const Args& p, hipStream_t stream) {
  constexpr int kRows = kThreads / TPR;
  // a launch has fewer than 2^32 threads
  const int64_t blocks = (p.rows_cap + kRows - 1) / kRows, most = (int64_t)1 << 23;
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0,
                       stream, p);
    return hipGetLastError();
  };
  return p.rows_cap * p.cols >= kStreamBytes
             ? run(quantize_int8_kernel<F16, TPR, NC, LONG, true>)
             : run(quantize_int8_kernel<F16, TPR, NC, LONG, false>);
}

// 256 threads a row from 2048 columns on: 114688 x 4096 227 us, with 512 threads 279;
// 32768 x 7168 121 us, with 512 threads 126, with 1024 166 (cached stores).
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
