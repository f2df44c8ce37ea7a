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
// A wave takes 512 columns of both halves, a lane 8 of each: 16-byte loads and stores, and
// the next 512 columns' loads before these are worked on.  A workgroup takes some whole rows, so
// that one XCD's L2 holds the lines of their scale bytes, of which a wave writes 16 bytes at a
// time, and its waves take the rows' chunks of 512 in turn.
#include "bsg_internal.h"
#include "mx_convert.h"

namespace bsg {

namespace {

constexpr int kChunk = 512;  // columns of a wave
constexpr int kMaxThreads = 1024;

// s(g).  The exponential's error is under 2^-16 of an s below 2^-64, which
// rounding to 16 bits hides, and 2^-22 around 1.  An s below 2^-126 (g under -87.3) is 0.
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

// A wave's chunks of its workgroup's rows: every waves-th of them, row after row.
struct Walk {
  int64_t row, last;
  int c, unit;             // chunk of the row, and of the workgroup's rows
  int chunks, waves, dr, dc;
  // block: the workgroup's rows are rows_each of them, from block * rows_each on.
  __device__ __forceinline__ void init(const Rows& rows, int n, int rows_each, int64_t block) {
    unit = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    waves = (int)(blockDim.x >> 6);
    chunks = n;
    dr = waves / n;
    dc = waves - dr * n;
    const int64_t first = rows.first + block * rows_each;
    last = first + rows_each < rows.last ? first + rows_each : rows.last;
    const int r = unit / n;
    row = first + r;
    c = unit - r * n;
  }
  __device__ __forceinline__ bool here() const { return row < last; }
  __device__ __forceinline__ void next() {
    unit += waves;
    row += dr;
    c += dc;
    if (c >= chunks) {
      c -= chunks;
      ++row;
    }
  }
};

// STREAM: past the caches, for outputs that would be written back from the last-level cache (256
// MiB) while the next call's data comes in.  us without and with it, calls in a row into four
// sets of outputs: 67 MB (16384 x 2048 forward) 46 and 50, 101 MB (8192 x 2048 backward, all
// outputs) 34.3 and 33.0, 134 MB (16384 x 4096 forward) 98 and 94, 266 MB (32000 x 2080
// backward) 99 and 93, 470 MB (16384 x 14336 forward) 332 and 308.  (Into the same outputs every
// time 266 MB take 82 without it: what the cache holds is written over.)
template <bool STREAM, typename T>
__device__ __forceinline__ void store(void* to, const T& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<T*>(to));
  else *reinterpret_cast<T*>(to) = v;
}

template <bool F16, bool STREAM>
__device__ __forceinline__ void store8(uint16_t* to, const float (&v)[8]) {
  store<STREAM>(to, v4i{(int)pack16<F16>(v[0], v[1]), (int)pack16<F16>(v[2], v[3]),
                        (int)pack16<F16>(v[4], v[5]), (int)pack16<F16>(v[6], v[7])});
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
  int G, rows_each;
};

template <bool F16, bool KEEP, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void swiglu_kernel(Fwd p) {
  const Rows rows = live_rows(p.offsets, p.G, p.rows_cap, p.status);
  const int lane = threadIdx.x & 63;
  const int f = (int)p.f;
  Walk at;
  v4i next_g, next_u;
  float next_w = 1.0f;
  const auto load = [&]() {
    next_g = next_u = v4i{0, 0, 0, 0};
    if (!at.here()) return;
    const int col = at.c * kChunk + 8 * lane;
    if (col < f) {  // of four lanes or none: f is a multiple of 32
      const uint16_t* src = p.h + at.row * p.ldh + col;
      next_g = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(src));
      next_u = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(src + f));
    }
    if (p.w != nullptr) next_w = p.w[at.row];
  };
  for (int64_t block = blockIdx.x; block * p.rows_each < rows.last - rows.first;
       block += gridDim.x) {
    at.init(rows, (f + kChunk - 1) / kChunk, p.rows_each, block);
    load();
    while (at.here()) {
      const v4i g = next_g, u = next_u;
      const float w = next_w;
      const int64_t row = at.row;
      const int col = at.c * kChunk + 8 * lane;
      const bool here = col < f;
      at.next();
      load();
      if constexpr (KEEP) {
        const uint32_t ag = block_amax(g), au = block_amax(u);
        const uint32_t bg = scale_byte<F16>(ag), bu = scale_byte<F16>(au);
        const v2i qg = codes8<F16>(g, bg), qu = codes8<F16>(u, bu);
        if (here) {
          uint8_t* dst = p.data + row * 2 * p.f + col;
          store<true>(dst, qg);  // not read before the backward pass
          store<true>(dst + f, qu);
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
      if (here) store8<F16, STREAM>(p.y + row * p.ldy + col, y);
    }
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
  int G, rows_each;
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

// ROWSUM: dw of the rows, added up in one order: a lane's terms of a chunk, the lanes, and when
// the rows are done their chunks.
constexpr int kMaxUnits = 2048;  // of a workgroup, with ROWSUM

template <bool F16, bool ROWSUM, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void swiglu_backward_kernel(Bwd p) {
  __shared__ float part[ROWSUM ? kMaxUnits : 1];
  const Rows rows = live_rows(p.offsets, p.G, p.rows_cap, p.status);
  const int lane = threadIdx.x & 63;
  const int f = (int)p.f;
  Walk at;
  struct Kept {
    v2i g, u;
    v4i dy;
    uint32_t bg, bu;
    float w;
  } next;
  next.w = 1.0f;
  const auto load = [&]() {
    if (!at.here()) return;
    const int col = at.c * kChunk + 8 * lane;
    if (col < f) {
      const uint8_t* src = p.data + at.row * 2 * p.f + col;
      next.g = __builtin_nontemporal_load(reinterpret_cast<const v2i*>(src));
      next.u = __builtin_nontemporal_load(reinterpret_cast<const v2i*>(src + f));
      const uint8_t* sc = p.scales + at.row * (p.f / 16) + col / 32;
      next.bg = sc[0];
      next.bu = sc[f / 32];
      next.dy = __builtin_nontemporal_load(
          reinterpret_cast<const v4i*>(p.dy + at.row * p.lddy + col));
    }
    if (p.w != nullptr) next.w = p.w[at.row];
  };
  for (int64_t block = blockIdx.x; block * p.rows_each < rows.last - rows.first;
       block += gridDim.x) {
    at.init(rows, (f + kChunk - 1) / kChunk, p.rows_each, block);
    load();
    while (at.here()) {
      const Kept k = next;
      const int64_t row = at.row;
      const int col = at.c * kChunk + 8 * lane, unit = at.unit;
      at.next();
      load();
      float dw = 0.0f;
      if (col < f) {
        float g[8], u[8], dg[8], du[8], y[8];
        decode8(k.g, k.bg, g);
        decode8(k.u, k.bu, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = sigmoid(g[e]), act = g[e] * s, dy = elem<F16>(k.dy, e);
          if constexpr (ROWSUM) dw += dy * act * u[e];
          const float dyw = dy * k.w;
          du[e] = dyw * act;
          dg[e] = dyw * u[e] * (s * fmaf(g[e], 1.0f - s, 1.0f));
          y[e] = k.w * act * u[e];
        }
        store8<F16, STREAM>(p.dh + row * p.lddh + col, dg);
        store8<F16, STREAM>(p.dh + row * p.lddh + f + col, du);
        if (p.y != nullptr) store8<F16, STREAM>(p.y + row * p.ldy + col, y);
      }
      if constexpr (ROWSUM) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) dw += __shfl_xor(dw, d, 64);
        if (lane == 0) part[unit] = dw;
      }
    }
    if constexpr (ROWSUM) {
      __syncthreads();
      const int64_t first = rows.first + block * p.rows_each;
      for (int r = (int)(threadIdx.x >> 6); first + r < at.last; r += at.waves) {
        float dw = 0.0f;
        for (int c = lane; c < at.chunks; c += 64) dw += part[r * at.chunks + c];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) dw += __shfl_xor(dw, d, 64);
        if (lane == 0) p.dw[first + r] = dw;
      }
      __syncthreads();  // the parts are read before the next rows'
    }
  }
}

// Workgroups of 16 waves where there is work for the chip in them (4 where not), and as many
// rows in each as give a wave some kRounds chunks.  16384 x 14336, forward and backward, and
// 32000 x 2080 backward (cached stores, the same outputs every time), us: 16 waves and 2 chunks
// each 306, 391 and 83, 3 chunks 307, 392 and 82 (6.2, 6.0 and 6.5 TB/s), 5 chunks 323, 402 and
// 84, 8 chunks 344, 431 and 86; 4 waves 348, 441 and 87.
// Less work than the chip takes at once, rows of more than 4 chunks, us with 16 and with 4 waves,
// forward and backward in a graph: 64 x 14336 5.1 and 5.7 against 7.7 and 8.0, 64 x 8192 4.1 and 4.7
// against 5.2 and 5.7, 1 x 2560 2.8 and 3.4 against 3.2 and 3.7.  Up to 8 chunks 4 waves win from some
// rows on (64 x 4096 3.6 and 4.2 against 3.9 and 4.6), and many rows' backward pass does at any
// length (1024 x 2560 6.5 against 9.1, 400 x 8192 8.0 against 9.1).
constexpr int64_t kRounds = 3;

struct Shape {
  int rows_each;
  unsigned grid, block;
};
Shape shape_of(int64_t rows_cap, int64_t f) {
  const int64_t chunks = (f + kChunk - 1) / kChunk, units = rows_cap * chunks;
  const int64_t slots = 32 * (int64_t)device_cu_count();  // waves on the chip
  const int64_t waves = units >= slots || chunks > 4 ? 16 : 4;
  int64_t rounds = units / slots;
  rounds = rounds < 1 ? 1 : rounds > kRounds ? kRounds : rounds;
  int64_t each = waves * rounds / chunks;
  if (each < 1) each = 1;
  if (each * chunks > kMaxUnits) each = kMaxUnits / chunks;
  // a launch has fewer than 2^32 threads
  const int64_t groups = (rows_cap + each - 1) / each, most = (int64_t)1 << 20;
  return {(int)each, (unsigned)(groups < most ? groups : most), (unsigned)(64 * waves)};
}

constexpr int64_t kStreamBytes = (int64_t)96 << 20;

template <typename K, typename P>
hipError_t run(K kernel, P p, hipStream_t stream) {
  const Shape s = shape_of(p.rows_cap, p.f);
  p.rows_each = s.rows_each;
  hipLaunchKernelGGL(kernel, dim3(s.grid), dim3(s.block), 0, stream, p);
  return hipGetLastError();
}

template <bool F16, bool KEEP>
hipError_t launch_forward(const Fwd& p, hipStream_t stream) {
  if (2 * p.rows_cap * p.f >= kStreamBytes) return run(swiglu_kernel<F16, KEEP, true>, p, stream);
  return run(swiglu_kernel<F16, KEEP, false>, p, stream);
}

template <bool F16, bool ROWSUM>
hipError_t launch_backward(const Bwd& p, hipStream_t stream) {
  if ((p.y != nullptr ? 6 : 4) * p.rows_cap * p.f >= kStreamBytes)
    return run(swiglu_backward_kernel<F16, ROWSUM, true>, p, stream);
  return run(swiglu_backward_kernel<F16, ROWSUM, false>, p, stream);
}

}  // namespace

hipError_t launch_swiglu_checkpoint(int f16, const void* h, int64_t ldh, const float* w, int G,
                                    const int64_t* offsets, int64_t rows_cap, int64_t f, void* y,
                                    int64_t ldy, uint8_t* data, uint8_t* scales, uint32_t* status,
                                    hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const Fwd p{static_cast<const uint16_t*>(h), ldh, w, offsets, rows_cap, f,
              static_cast<uint16_t*>(y), ldy, data, scales, status, G, 0};
  if (data != nullptr)
    return f16 ? launch_forward<true, true>(p, stream) : launch_forward<false, true>(p, stream);
  return f16 ? launch_forward<true, false>(p, stream) : launch_forward<false, false>(p, stream);
}

hipError_t launch_swiglu_checkpoint_backward(int f16, const uint8_t* data, const uint8_t* scales,
                                             const float* w, const void* dy, int64_t lddy, int G,
                                             const int64_t* offsets, int64_t rows_cap, int64_t f,
                                             void* dh, int64_t lddh, void* y, int64_t ldy,
                                             float* dw, uint32_t* status, hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const Bwd p{data, scales, w, static_cast<const uint16_t*>(dy), lddy, offsets, rows_cap, f,
              static_cast<uint16_t*>(dh), lddh, static_cast<uint16_t*>(y), ldy, dw, status, G, 0};
  if (dw != nullptr)
    return f16 ? launch_backward<true, true>(p, stream) : launch_backward<false, true>(p, stream);
  return f16 ? launch_backward<true, false>(p, stream) : launch_backward<false, false>(p, stream);
}

}  // namespace bsg
