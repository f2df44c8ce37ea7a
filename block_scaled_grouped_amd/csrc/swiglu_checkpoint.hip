// The gated activation between an expert's two products, kept in 8 bits for the backward
// pass.  h = [g | u] is the first product's output, w a weight of the row (or 1):
//
//   y = w g s(g) u,   s(g) = 1 / (1 + exp(-g))
//
// and what is kept of h is its MXFP8 form: E4M3 elements and one E8M0 scale for each 32
// along the row, the bytes of the rowwise quantize (scales row by row here: no matrix
// instruction reads them).  Backwards, at the kept g and u:
//
//   dg = dy w u s (1 + g (1 - s)),  du = dy w g s,  dw = sum over the row of dy g s u
//
// and y again, for the second product's weight gradient.
//
// HBM bound: forward 8 bytes and 1/16 an element of y, backward 10 and 1/16 (8 without y).
// A wave takes 512 columns of both halves, a lane 8 of each: 16-byte loads and stores.
#include "bsg_internal.h"
#include "mx_convert.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 512;  // columns of a wave

// g s(g) and s(g).  The exponential's error is under 2^-16 of an s below 2^-64, which
// rounding to 16 bits hides, and 2^-22 around 1.
__device__ __forceinline__ float sigmoid(float g) {
  const float e = __builtin_amdgcn_exp2f(g * -1.44269502162933349609375f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

template <bool F16>
__device__ __forceinline__ float elem(const v4i& v, int e) {
  const uint32_t w = (uint32_t)v[e >> 1];
  if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)(e & 1 ? w >> 16 : w));
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

// The largest magnitude bits of a block: of 8 values here and in the three lanes beside.
__device__ __forceinline__ uint32_t block_amax(const v4i& v) {
  uint32_t m = amax_fold(amax2(amax2((uint32_t)v[0], (uint32_t)v[1]),
                               amax2((uint32_t)v[2], (uint32_t)v[3])));
  m = max(m, dpp_xor1(m));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
}

// The scale byte of a block whose largest magnitude has these 16 bits.
template <bool F16>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if constexpr (F16) {
    // fp16's subnormal numbers are normal in float32
    const uint32_t e =
        __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)amax)) >> 23;
    return e > 8 ? e - 8 : 0u;
  }
  return e8m0_from_amax_bits(amax);
}

template <bool F16>
__device__ __forceinline__ v2i codes8(const v4i& v, uint32_t byte) {
  const float scale = e8m0_scale(byte);
  if constexpr (!F16) {
    const uint2 q = cvt8(make_uint4((uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]),
                         scale);
    return v2i{(int)q.x, (int)q.y};
  } else {
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    v2i q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int lo = v[2 * h], hi = v[2 * h + 1];
      v2s r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(v2s{0, 0}, __builtin_bit_cast(v2h, lo), scale,
                                                       false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(v2h, hi), scale, true);
      q[h] = (int)fp8_saturate(__builtin_bit_cast(uint32_t, r));
    }
    return q;
  }
}

// Rows [first, last) of the groups, inside of the buffers.
struct Rows {
  int64_t first, last;
};
__device__ __forceinline__ Rows live_rows(const int64_t* offsets, int G, int64_t rows_cap,
                                          uint32_t* status) {
  Rows r{offsets[0], offsets[G]};
  const uint32_t bad = (r.first < 0 || r.last < r.first ? kDevNegativeSize : 0u) |
                       (r.last > rows_cap || r.first > rows_cap ? kDevOverCapacity : 0u);
  if (bad != 0 && blockIdx.x == 0 && threadIdx.x == 0) dev_status_or(status, bad);
  if (r.first < 0) r.first = 0;
  if (r.last > rows_cap) r.last = rows_cap;
  return r;
}

struct Fwd {
  const uint16_t* h;
  int64_t ldh;
  const float* w;
  const int64_t* offsets;
  int64_t rows_cap, f;
  uint16_t* y;
  int64_t ldy;
  uint8_t* data;
  uint8_t* scales;
  uint32_t* status;
  int G;
};

template <bool F16, bool KEEP>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(Fwd p) {
  const Rows rows = live_rows(p.offsets, p.G, p.rows_cap, p.status);
  const int lane = threadIdx.x & 63;
  const int f = (int)p.f, chunks = (f + kChunk - 1) / kChunk;
  const int64_t units = (rows.last - rows.first) * chunks;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); unit < units;
       unit += stride) {
    const int64_t row = rows.first + unit / chunks;
    const int col = (int)(unit % chunks) * kChunk + 8 * lane;
    const bool here = col < f;  // of four lanes or none: f is a multiple of 32
    v4i g = v4i{0, 0, 0, 0}, u = v4i{0, 0, 0, 0};
    if (here) {
      const uint16_t* src = p.h + row * p.ldh + col;
      g = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(src));
      u = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(src + f));
    }
    const float w = p.w != nullptr ? p.w[row] : 1.0f;
    if constexpr (KEEP) {
      const uint32_t ag = block_amax(g), au = block_amax(u);
      const uint32_t bg = scale_byte<F16>(ag), bu = scale_byte<F16>(au);
      const v2i qg = codes8<F16>(g, bg), qu = codes8<F16>(u, bu);
      if (here) {
        uint8_t* dst = p.data + row * 2 * p.f + col;
        *reinterpret_cast<v2i*>(dst) = qg;
        *reinterpret_cast<v2i*>(dst + f) = qu;
        if ((lane & 3) == 0) {
          uint8_t* sc = p.scales + row * (p.f / 16) + col / 32;
          sc[0] = (uint8_t)bg;
          sc[f / 32] = (uint8_t)bu;
        }
      }
      if (__any(max(ag, au) >= (F16 ? 0x7c00u : 0x7f80u)) && lane == 0)
        dev_status_or(p.status, kDevNonFinite);
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = elem<F16>(g, e);
      y[e] = w * (x * sigmoid(x)) * elem<F16>(u, e);
    }
    if (here)
      *reinterpret_cast<v4i*>(p.y + row * p.ldy + col) =
          v4i{(int)pack16<F16>(y[0], y[1]), (int)pack16<F16>(y[2], y[3]),
              (int)pack16<F16>(y[4], y[5]), (int)pack16<F16>(y[6], y[7])};
  }
}

struct Bwd {
  const uint8_t* data;
  const uint8_t* scales;
  const float* w;
  const uint16_t* dy;
  int64_t lddy;
  const int64_t* offsets;
  int64_t rows_cap, f;
  uint16_t* dh;
  int64_t lddh;
  uint16_t* y;
  int64_t ldy;
  float* dw;
  uint32_t* status;
  int G;
};

// 8 kept values of a half.
__device__ __forceinline__ void decode8(const v2i& q, uint32_t byte, float (&v)[8]) {
  const float scale = e8m0_scale(byte);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)q[h], scale, false);
    const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((uint32_t)q[h], scale, true);
    v[4 * h] = a[0];
    v[4 * h + 1] = a[1];
    v[4 * h + 2] = b[0];
    v[4 * h + 3] = b[1];
  }
}

// One wave's 512 columns of a row; returns its share of dw.
template <bool F16>
__device__ __forceinline__ float backward_chunk(const Bwd& p, int64_t row, int col, float w) {
  const int f = (int)p.f;
  float dw = 0.0f;
  if (col < f) {
    const uint8_t* src = p.data + row * 2 * p.f + col;
    const v2i qg = __builtin_nontemporal_load(reinterpret_cast<const v2i*>(src));
    const v2i qu = __builtin_nontemporal_load(reinterpret_cast<const v2i*>(src + f));
    const uint8_t* sc = p.scales + row * (p.f / 16) + col / 32;
    const uint32_t bg = sc[0], bu = sc[f / 32];
    const v4i d = __builtin_nontemporal_load(
        reinterpret_cast<const v4i*>(p.dy + row * p.lddy + col));
    float g[8], u[8], dg[8], du[8], y[8];
    decode8(qg, bg, g);
    decode8(qu, bu, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sigmoid(g[e]), act = g[e] * s, dy = elem<F16>(d, e);
      dw += dy * act * u[e];
      const float dyw = dy * w;
      du[e] = dyw * act;
      dg[e] = dyw * u[e] * (s * fmaf(g[e], 1.0f - s, 1.0f));
      y[e] = w * act * u[e];
    }
    const auto store = [&](uint16_t* at, const float (&v)[8]) {
      *reinterpret_cast<v4i*>(at) =
          v4i{(int)pack16<F16>(v[0], v[1]), (int)pack16<F16>(v[2], v[3]),
              (int)pack16<F16>(v[4], v[5]), (int)pack16<F16>(v[6], v[7])};
    };
    store(p.dh + row * p.lddh + col, dg);
    store(p.dh + row * p.lddh + f + col, du);
    if (p.y != nullptr) store(p.y + row * p.ldy + col, y);
  }
  return dw;
}

// ROWSUM: a workgroup of WPR waves a row adds up dw in one order; else every wave takes
// the next 512 columns wherever they lie.
template <bool F16, bool ROWSUM, int WPR>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(Bwd p) {
  const Rows rows = live_rows(p.offsets, p.G, p.rows_cap, p.status);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int f = (int)p.f, chunks = (f + kChunk - 1) / kChunk;
  if constexpr (!ROWSUM) {
    const int64_t units = (rows.last - rows.first) * chunks;
    const int64_t stride = (int64_t)gridDim.x * (kThreads / 64);
    for (int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + wave; unit < units;
         unit += stride) {
      const int64_t row = rows.first + unit / chunks;
      backward_chunk<F16>(p, row, (int)(unit % chunks) * kChunk + 8 * lane,
                          p.w != nullptr ? p.w[row] : 1.0f);
    }
  } else {
    constexpr int kRows = kThreads / 64 / WPR;
    __shared__ float part[2][kThreads / 64];
    const int64_t count = rows.last - rows.first;
    int turn = 0;
    for (int64_t r = (int64_t)blockIdx.x * kRows; r < count; r += (int64_t)gridDim.x * kRows) {
      const int64_t row = rows.first + r + wave / WPR;
      float dw = 0.0f;
      if (row < rows.last) {
        const float w = p.w != nullptr ? p.w[row] : 1.0f;
        for (int c = wave % WPR; c < chunks; c += WPR)
          dw += backward_chunk<F16>(p, row, c * kChunk + 8 * lane, w);
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) dw += __shfl_xor(dw, d, 64);
      if constexpr (WPR > 1) {
        if (lane == 0) part[turn][wave] = dw;
        __syncthreads();
        dw = 0.0f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) dw += part[turn][wave / WPR * WPR + i];
        turn ^= 1;  // the next row's parts go elsewhere: one barrier a row
      }
      if (lane == 0 && wave % WPR == 0 && row < rows.last) p.dw[row] = dw;
    }
  }
}

unsigned grid_for(int64_t workgroups) {
  const int64_t cap = 32 * (int64_t)device_cu_count();
  return (unsigned)(workgroups < cap ? workgroups : cap);
}

template <bool F16>
hipError_t launch_backward(const Bwd& p, hipStream_t stream) {
  const int64_t chunks = (p.f + kChunk - 1) / kChunk;
  const auto run = [&](auto kernel, int64_t workgroups) {
    hipLaunchKernelGGL(kernel, dim3(grid_for(workgroups)), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
  };
  if (p.dw == nullptr)
    return run(swiglu_backward_kernel<F16, false, 1>, (p.rows_cap * chunks + 3) / 4);
  if (chunks == 1) return run(swiglu_backward_kernel<F16, true, 1>, (p.rows_cap + 3) / 4);
  if (chunks == 2) return run(swiglu_backward_kernel<F16, true, 2>, (p.rows_cap + 1) / 2);
  return run(swiglu_backward_kernel<F16, true, 4>, p.rows_cap);
}

}  // namespace

hipError_t launch_swiglu_checkpoint(int f16, const void* h, int64_t ldh, const float* w, int G,
                                    const int64_t* offsets, int64_t rows_cap, int64_t f, void* y,
                                    int64_t ldy, uint8_t* data, uint8_t* scales, uint32_t* status,
                                    hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const Fwd p{static_cast<const uint16_t*>(h), ldh, w, offsets, rows_cap, f,
              static_cast<uint16_t*>(y), ldy, data, scales, status, G};
  const dim3 grid(grid_for((rows_cap * ((f + kChunk - 1) / kChunk) + 3) / 4));
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
  };
  if (data != nullptr) return f16 ? run(swiglu_kernel<true, true>) : run(swiglu_kernel<false, true>);
  return f16 ? run(swiglu_kernel<true, false>) : run(swiglu_kernel<false, false>);
}

hipError_t launch_swiglu_checkpoint_backward(int f16, const uint8_t* data, const uint8_t* scales,
                                             const float* w, const void* dy, int64_t lddy, int G,
                                             const int64_t* offsets, int64_t rows_cap, int64_t f,
                                             void* dh, int64_t lddh, void* y, int64_t ldy,
                                             float* dw, uint32_t* status, hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const Bwd p{data, scales, w, static_cast<const uint16_t*>(dy), lddy, offsets, rows_cap, f,
              static_cast<uint16_t*>(dh), lddh, static_cast<uint16_t*>(y), ldy, dw, status, G};
  return f16 ? launch_backward<true>(p, stream) : launch_backward<false>(p, stream);
}

}  // namespace bsg
