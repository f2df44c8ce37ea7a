// Grouped products of 16-bit operands (bf16 or fp16) with FP32 accumulation.
//
//   FPROP_TN:  Y[r, :]  = A[r, :] B_g^T        r in group g, contraction k
//   DGRAD_NN:  Y[r, :]  = A[r, :] B_g          r in group g, contraction k
//   WGRAD_NT:  Y_g      = C_g + A_g^T B_g      contraction over the group's rows
//
// and, beside a projection shared by all rows, the low-rank product of each
// row's own adapter (LORA): Y[r, :] = A[r, :] B^T + low[r, :] U_a^T.
//
// Every tile is one contraction of an A tile and a B tile, each of which lies in
// memory either with the contraction innermost or with its rows innermost.
#include "bsg_internal.h"
#include "store_tile.h"

namespace bsg {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int BM = 128, BN = 128, BK = 32;
constexpr int kThreads = 256;
constexpr int kLdsRow = BK + 8;  // elements
constexpr int kSuperM = 4, kSuperN = 8;

struct Args16 {
  const uint16_t* a;
  const uint16_t* b;
  const int64_t* offsets;
  const char* c;
  char* out;
  int64_t lda, ldb, stride_b, ldo, stride_o;  // elements
  int64_t rows_cap, n, k;
  uint32_t* status;
  int G, out_f32;
  // LORA
  const uint16_t* low;      // [rows_cap, 2 r]: high and low halves of the scaled X A^T
  const uint16_t* up;       // [adapters, n, r]
  const int32_t* adapter;   // [G], negative: none
  int num_adapters, r;
};

struct Tile16 {
  const uint16_t* a;
  const uint16_t* b;
  int64_t lda, ldb;
  int a_rows, b_rows;
  int64_t kl;
  char* out;
  const char* c;
  int ldo;
  int out_rows, out_cols;
};

struct Sched16 {
  int64_t off[kMaxGroups + 1];
  int32_t cnt[kMaxGroups];
  int32_t pre[kMaxGroups + 1];
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

template <bool F16>
__device__ __forceinline__ v16f mfma16(const v4i& x, const v4i& y, const v16f& acc) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, x),
                                                  __builtin_bit_cast(v8h, y), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x),
                                                   __builtin_bit_cast(v8bf, y), acc, 0, 0, 0);
}

// Copies a 128 x 32 operand tile into LDS with the contraction innermost.  Rows
// and contraction indexes past the operand's are zeros.
template <bool TR>
__device__ __forceinline__ void stage_tile(uint16_t (*s)[kLdsRow], const uint16_t* src, int64_t ld,
                                           int rows, int64_t k0, int64_t kl) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int id = threadIdx.x + q * kThreads;
    v4i v = v4i{0, 0, 0, 0};
    if constexpr (!TR) {
      const int row = id >> 2, kc = (id & 3) * 8;
      if (row < rows && k0 + kc < kl)
        v = *reinterpret_cast<const v4i*>(src + (int64_t)row * ld + k0 + kc);
      *reinterpret_cast<v4i*>(&s[row][kc]) = v;
    } else {
      const int kr = id >> 4, row = (id & 15) * 8;
      if (row < rows && k0 + kr < kl)
        v = *reinterpret_cast<const v4i*>(src + (k0 + kr) * ld + row);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        s[row + e][kr] = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
    }
  }
}

template <bool F16, bool TA, bool TB>
__device__ __forceinline__ void contract(uint16_t (*sa)[kLdsRow], uint16_t (*sb)[kLdsRow],
                                         const Tile16& t, int64_t kl, v16f (&acc)[2][2]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int r = lane & 31, h = lane >> 5;
  for (int64_t k0 = 0; k0 < kl; k0 += BK) {
    stage_tile<TA>(sa, t.a, t.lda, t.a_rows, k0, kl);
    stage_tile<TB>(sb, t.b, t.ldb, t.b_rows, k0, kl);
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < BK; ks += 16) {
      v4i fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const v4i*>(&sa[(w >> 1) * 64 + 32 * i + r][ks + 8 * h]);
        fb[i] = *reinterpret_cast<const v4i*>(&sb[(w & 1) * 64 + 32 * i + r][ks + 8 * h]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma16<F16>(fb[j], fa[i], acc[i][j]);
    }
    __syncthreads();
  }
}

// One 32 x 32 block with C added in float32 before the one rounding.
template <bool F32, bool F16>
__device__ __forceinline__ void store_block_c(const v16f& acc, __amdgpu_buffer_rsrc_t ro,
                                              __amdgpu_buffer_rsrc_t rc, int ldo, int row, int col0,
                                              int out_cols) {
  constexpr int esz = F32 ? 4 : 2;
  int off[4];
  float c[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int col = col0 + 8 * q;
    off[q] = col < out_cols ? (row * ldo + col) * esz : (int)kDropped;
    if constexpr (F32) {
      const v4i v = __builtin_amdgcn_raw_buffer_load_b128(rc, off[q], 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[4 * q + e] = __int_as_float(v[e]);
    } else {
      const v2i v = __builtin_amdgcn_raw_buffer_load_b64(rc, off[q], 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bits = ((uint32_t)v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
        c[4 * q + e] = F16 ? (float)__builtin_bit_cast(_Float16, (unsigned short)bits)
                           : bf16_to_f32(bits);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = acc[4 * q + e] + c[4 * q + e];
    if constexpr (F32) {
      __builtin_amdgcn_raw_buffer_store_b128(
          (v4i){__float_as_int(y[0]), __float_as_int(y[1]), __float_as_int(y[2]),
                __float_as_int(y[3])},
          ro, off[q], 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b64(
          (v2i){(int)pack16<F16>(y[0], y[1]), (int)pack16<F16>(y[2], y[3])}, ro, off[q], 0, 0);
    }
  }
}

template <int MODE, bool F16, bool LORA>
__global__ __launch_bounds__(kThreads) void gemm16_kernel(Args16 p) {
  constexpr bool kWgrad = MODE == 1;
  __shared__ __attribute__((aligned(16))) uint16_t sa[BM][kLdsRow];
  __shared__ __attribute__((aligned(16))) uint16_t sb[BN][kLdsRow];
  __shared__ Sched16 sm;
  const int G = p.G, tid = threadIdx.x;
  load_offsets_clamped(p.offsets, G, p.rows_cap, sm.off, blockIdx.x == 0 ? p.status : nullptr);
  const int64_t ntn = (p.n + BN - 1) / BN;
  const int items = LORA ? 1 : G;
  if constexpr (LORA) {
    // all rows of all requests are one run of rows of the shared projection
    if (tid == 0) {
      const int64_t m = sm.off[G] - sm.off[0];
      sm.cnt[0] = (int32_t)(((m > 0 ? m : 0) + BM - 1) / BM * ntn);
    }
  } else {
    for (int g = tid; g < G; g += kThreads)
      sm.cnt[g] = (int32_t)(kWgrad ? ((p.n + BM - 1) / BM) * ((p.k + BN - 1) / BN)
                                   : ((group_extent(sm.off, g) + BM - 1) / BM) * ntn);
  }
  __syncthreads();
  wave0_exclusive_scan(sm.cnt, items, sm.pre);
  __syncthreads();
  const int total = sm.pre[items];
  const int esz = p.out_f32 ? 4 : 2;
  const int lane = tid & 63, w = tid >> 6;

  for (int tile = xcd_slot(); tile < total; tile += gridDim.x) {
    const int g = find_group(sm.pre, items, tile);
    const int local = tile - sm.pre[g];
    const int64_t m = LORA ? sm.off[G] - sm.off[0] : group_extent(sm.off, g);
    Tile16 t;
    int mt, nt;
    if constexpr (!kWgrad) {
      super_tile<kSuperM, kSuperN>(local, (int)((m + BM - 1) / BM), (int)ntn, mt, nt);
      const int64_t row0 = sm.off[g] + (int64_t)mt * BM, n0 = (int64_t)nt * BN;
      t.a = p.a + row0 * p.lda;
      t.lda = p.lda;
      t.b = p.b + (LORA ? 0 : g * p.stride_b) + (MODE == 0 ? n0 * p.ldb : n0);
      t.ldb = p.ldb;
      const int64_t rv = sm.off[g] + m - row0, cv = p.n - n0;
      t.a_rows = (int)(rv < BM ? rv : BM);
      t.b_rows = (int)(cv < BN ? cv : BN);
      t.kl = p.k;
      const int64_t o = (row0 * p.ldo + n0) * esz;
      t.out = p.out + o;
      t.c = p.c != nullptr ? p.c + o : nullptr;
    } else {
      super_tile<kSuperM, kSuperN>(local, (int)((p.n + BM - 1) / BM), (int)((p.k + BN - 1) / BN),
                                   mt, nt);
      const int64_t i0 = (int64_t)mt * BM, j0 = (int64_t)nt * BN;
      t.a = p.a + sm.off[g] * p.lda + i0;
      t.b = p.b + sm.off[g] * p.ldb + j0;
      t.lda = p.lda;
      t.ldb = p.ldb;
      const int64_t rv = p.n - i0, cv = p.k - j0;
      t.a_rows = (int)(rv < BM ? rv : BM);
      t.b_rows = (int)(cv < BN ? cv : BN);
      t.kl = m;
      const int64_t o = (g * p.stride_o + i0 * p.ldo + j0) * esz;
      t.out = p.out + o;
      t.c = p.c != nullptr ? p.c + o : nullptr;
    }
    t.ldo = (int)p.ldo;
    t.out_rows = t.a_rows;
    t.out_cols = t.b_rows;

    v16f acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = v16f{};
    contract<F16, kWgrad, MODE != 0>(sa, sb, t, t.kl, acc);
    if constexpr (LORA) {
      const int64_t row0 = sm.off[0] + (int64_t)mt * BM, n0 = (int64_t)nt * BN;
      for (int q = 0; q < G; ++q) {
        int64_t lo = sm.off[q] - row0, hi = sm.off[q + 1] - row0;
        if (lo < 0) lo = 0;
        if (hi > t.a_rows) hi = t.a_rows;
        const int ad = p.adapter[q];
        if (lo >= hi || ad < 0 || ad >= p.num_adapters) continue;
        Tile16 u = t;
        u.ldb = p.r;
        u.lda = 2 * p.r;
        u.b = p.up + ((int64_t)ad * p.n + n0) * p.r;
        u.a = p.low + row0 * 2 * p.r;
        // the product of the tile's rows with this adapter, kept for the rows
        // of its own requests only: what an adapter holds (infinities, NaN)
        // never reaches a row of another
        v16f one[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) one[i][j] = v16f{};
        contract<F16, false, false>(sa, sb, u, p.r, one);
        u.a += p.r;
        contract<F16, false, false>(sa, sb, u, p.r, one);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = (w >> 1) * 64 + 32 * i + (lane & 31);
          if (row >= lo && row < hi) {
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] += one[i][j];
          }
        }
      }
    }
    const __amdgpu_buffer_rsrc_t ro = make_rsrc(t.out, (int64_t)t.out_rows * t.ldo * esz);
    const __amdgpu_buffer_rsrc_t rc =
        make_rsrc(t.c, t.c != nullptr ? (int64_t)t.out_rows * t.ldo * esz : 0);
    const int row = (w >> 1) * 64 + (lane & 31), h = lane >> 5, col = (w & 1) * 64 + 4 * h;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ri = row + 32 * i, cj = col + 32 * j;
        if (t.c != nullptr) {
          if (p.out_f32) store_block_c<true, F16>(acc[i][j], ro, rc, t.ldo, ri, cj, t.out_cols);
          else store_block_c<false, F16>(acc[i][j], ro, rc, t.ldo, ri, cj, t.out_cols);
        } else {
          if (p.out_f32) store_block<true, true>(acc[i][j], ro, t.ldo, ri, cj, h, t.out_cols);
          else store_block<true, false, F16>(acc[i][j], ro, t.ldo, ri, cj, h, t.out_cols);
        }
      }
  }
}

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t b) {
  return F16 ? (float)__builtin_bit_cast(_Float16, b) : bf16_to_f32(b);
}

// s as the sum of two 16-bit values: the nearest one and the nearest to what is
// left (22 or 16 bits of s together).  The first is kept finite, so that a value
// past the type's range turns into an infinity in the second and not into the
// difference of two.
template <bool F16>
__device__ __forceinline__ void split16(float s, uint32_t& top, uint32_t& rest) {
  constexpr float kMax = F16 ? 65504.0f : 3.3895313892515355e38f;
  float c = s;
  if (s > kMax) c = kMax;
  if (s < -kMax) c = -kMax;
  top = pack16<F16>(c, c) & 0xffffu;
  const float left = s - to_f32<F16>((uint16_t)top);
  rest = pack16<F16>(left, left) & 0xffffu;
}

// low[t, 0..r) + low[t, r..2r) = scale_a X[t, :] A_a^T, one wavefront a value.
template <bool F16>
__global__ __launch_bounds__(kThreads) void lora_low_kernel(Args16 p, const uint16_t* down,
                                                            const float* scale, uint16_t* low) {
  __shared__ Sched16 sm;
  load_offsets_clamped(p.offsets, p.G, p.rows_cap, sm.off, nullptr);
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < p.G; g += kThreads)
      if (p.adapter[g] >= p.num_adapters) dev_status_or(p.status, kDevBadAdapter);
  const int64_t first = sm.off[0], last = sm.off[p.G];
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * (kThreads / 64);
  for (int64_t id = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
       id < (last - first) * p.r; id += waves) {
    const int64_t row = first + id / p.r;
    const int j = (int)(id % p.r);
    int g = 0, hi = p.G - 1;
    while (g < hi) {
      const int mid = (g + hi + 1) >> 1;
      if (sm.off[mid] <= row) g = mid; else hi = mid - 1;
    }
    const int ad = p.adapter[g];
    float s = 0.0f;
    if (ad >= 0 && ad < p.num_adapters) {
      const uint16_t* x = p.a + row * p.lda;
      const uint16_t* d = down + ((int64_t)ad * p.r + j) * p.k;
      for (int64_t i = lane; i < p.k; i += 64) s += to_f32<F16>(x[i]) * to_f32<F16>(d[i]);
      for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
      s *= scale[ad];
    }
    if (lane == 0) {
      uint32_t top, rest;
      split16<F16>(s, top, rest);
      low[row * 2 * p.r + j] = (uint16_t)top;
      low[row * 2 * p.r + p.r + j] = (uint16_t)rest;
    }
  }
}

}  // namespace

size_t gemm_16bit_workspace_bytes() { return 256; }

hipError_t launch_gemm_16bit(int mode, int f16, int G, const void* a, int64_t lda, const void* b,
                             int64_t ldb, int64_t stride_b, const int64_t* offsets,
                             int64_t rows_cap, int64_t n, int64_t k, const void* c, void* out,
                             int64_t ldo, int64_t stride_o, int out_f32, void* ws, uint32_t* status,
                             hipStream_t stream) {
  (void)ws;
  Args16 p{};
  p.a = static_cast<const uint16_t*>(a);
  p.b = static_cast<const uint16_t*>(b);
  p.offsets = offsets;
  p.c = static_cast<const char*>(c);
  p.out = static_cast<char*>(out);
  p.lda = lda; p.ldb = ldb; p.stride_b = stride_b; p.ldo = ldo; p.stride_o = stride_o;
  p.rows_cap = rows_cap; p.n = n; p.k = k;
  p.status = status;
  p.G = G; p.out_f32 = out_f32;
  int64_t bound;
  if (mode != 1) bound = ((rows_cap + BM - 1) / BM + G) * ((n + BN - 1) / BN);
  else bound = (int64_t)G * ((n + BM - 1) / BM) * ((k + BN - 1) / BN);
  int64_t grid = 4 * device_cu_count();
  if (bound < grid) grid = bound;
  if (grid <= 0) return hipSuccess;
  const dim3 gd((unsigned)grid), bd(kThreads);
  if (f16) {
    if (mode == 0) hipLaunchKernelGGL((gemm16_kernel<0, true, false>), gd, bd, 0, stream, p);
    else if (mode == 1) hipLaunchKernelGGL((gemm16_kernel<1, true, false>), gd, bd, 0, stream, p);
    else hipLaunchKernelGGL((gemm16_kernel<2, true, false>), gd, bd, 0, stream, p);
  } else {
    if (mode == 0) hipLaunchKernelGGL((gemm16_kernel<0, false, false>), gd, bd, 0, stream, p);
    else if (mode == 1) hipLaunchKernelGGL((gemm16_kernel<1, false, false>), gd, bd, 0, stream, p);
    else hipLaunchKernelGGL((gemm16_kernel<2, false, false>), gd, bd, 0, stream, p);
  }
  return hipGetLastError();
}

size_t lora_gemm_16bit_workspace_bytes(int64_t rows_cap, int64_t n, int64_t k, int64_t r) {
  (void)n;
  (void)k;
  return ((size_t)rows_cap * (size_t)r * 4 + 255) / 256 * 256 + 256;
}

hipError_t launch_lora_gemm_16bit(int f16, int G, const void* x, int64_t ldx, const void* w,
                                  int64_t ldw, const void* down, const void* up,
                                  int64_t num_adapters, int64_t r, const int64_t* offsets,
                                  const int32_t* adapter, const float* scale, int64_t rows_cap,
                                  int64_t n, int64_t k, void* out, int64_t ldo, int out_f32,
                                  void* ws, uint32_t* status, hipStream_t stream) {
  if (rows_cap <= 0) return hipSuccess;
  Args16 p{};
  p.a = static_cast<const uint16_t*>(x);
  p.b = static_cast<const uint16_t*>(w);
  p.offsets = offsets;
  p.out = static_cast<char*>(out);
  p.lda = ldx; p.ldb = ldw; p.ldo = ldo;
  p.rows_cap = rows_cap; p.n = n; p.k = k;
  p.status = status;
  p.G = G; p.out_f32 = out_f32;
  p.low = static_cast<uint16_t*>(ws);
  p.up = static_cast<const uint16_t*>(up);
  p.adapter = adapter;
  p.num_adapters = (int)num_adapters;
  p.r = (int)r;
  const dim3 bd(kThreads);
  const unsigned cus = (unsigned)device_cu_count();
  const uint16_t* d = static_cast<const uint16_t*>(down);
  uint16_t* low = static_cast<uint16_t*>(ws);
  int64_t grid = 4 * (int64_t)cus;
  const int64_t bound = ((rows_cap + BM - 1) / BM) * ((n + BN - 1) / BN);
  if (bound < grid) grid = bound;
  if (f16) {
    hipLaunchKernelGGL(lora_low_kernel<true>, dim3(8 * cus), bd, 0, stream, p, d, scale, low);
    hipLaunchKernelGGL((gemm16_kernel<0, true, true>), dim3((unsigned)grid), bd, 0, stream, p);
  } else {
    hipLaunchKernelGGL(lora_low_kernel<false>, dim3(8 * cus), bd, 0, stream, p, d, scale, low);
    hipLaunchKernelGGL((gemm16_kernel<0, false, true>), dim3((unsigned)grid), bd, 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace bsg
