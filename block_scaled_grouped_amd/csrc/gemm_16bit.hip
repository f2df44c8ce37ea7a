// 16-bit grouped products: which form runs, and the first product of the adapters.
#include "gemm_16bit.h"

namespace bsg {

using namespace g16;

namespace {

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

// low[t, 0..r) + low[t, r..2r) = scale_a X[t, :] A_a^T.
//
// A workgroup of eight waves takes 32 consecutive rows, 64 rank columns and one
// of the adapters that occur in those rows; the waves take turns at the
// contraction's runs of 64 (a 128-byte line of a row) and their sums are added
// through LDS in one order.  Rows of another adapter are computed too and not
// written.  Operands come straight from memory: X is read once an adapter and 64
// rank columns, and nothing is shared between waves that LDS could serve.
constexpr int kLowThreads = 512;
constexpr int kLowWaves = kLowThreads / 64;
constexpr int kLowRows = 32;

template <bool F16, int NB>  // 16 NB <= 64 rank columns a workgroup
__global__ __launch_bounds__(kLowThreads) void lora_low_kernel(Args p, const uint16_t* down,
                                                               const float* scale, uint16_t* low,
                                                               int turns) {
  __shared__ int64_t off[kMaxGroups + 1];
  __shared__ __attribute__((aligned(16))) v4f sums[kLowWaves][2][NB][64];
  load_offsets_clamped(p.offsets, p.G, p.rows_cap, off, nullptr);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int g = threadIdx.x; g < p.G; g += kLowThreads)
      if (p.adapter[g] >= p.num_adapters) dev_status_or(p.status, kDevBadAdapter);
  const int64_t first = uni64(off[0]), last = uni64(off[p.G]);
  const int lane = threadIdx.x & 63, w = uni((int)(threadIdx.x >> 6));
  const int r = lane & 15, q = lane >> 4, rank = p.r, k = (int)p.k;
  const int rank_blocks = (rank + 16 * NB - 1) / (16 * NB);
  const int64_t items = (last - first + kLowRows - 1) / kLowRows * rank_blocks * turns;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int turn0 = uni((int)(it % turns));
    const int j0 = uni((int)(it / turns % rank_blocks)) * (16 * NB);
    const int64_t row0 = first + it / turns / rank_blocks * kLowRows;
    // lane l: adapter of row l % 32
    const int64_t mine_row = row0 + (lane & 31);
    const int id = mine_row < last ? adapter_of(p, request_of(off, p.G, mine_row)) : -1;
    const uint16_t* x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = row0 + 16 * i + r;
      x[i] = p.a + (row < last ? row : last - 1) * p.lda + 8 * q;
    }
    uint32_t todo = (uint32_t)__ballot(id >= 0);
    int turn = 0;
    while (todo != 0) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
      const uint32_t own = (uint32_t)__ballot(id == a);
      todo &= ~own;
      const bool mine = turn == turn0;
      turn = turn + 1 == turns ? 0 : turn + 1;
      if (!mine) continue;
      const uint16_t* d[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        int j = j0 + 16 * b + r;
        if (j >= rank) j = rank - 1;  // such columns are not written
        d[b] = down + ((int64_t)a * rank + j) * p.k + 8 * q;
      }
      v4f acc[2][NB];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[i][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      // kRuns of the wave's runs are loaded before the first is used
      constexpr int kRuns = NB == 4 ? 2 : 4;
      for (int k0 = 64 * w; k0 < k; k0 += 64 * kLowWaves * kRuns) {
        v4i fx[2 * kRuns][2], fd[2 * kRuns][NB];
#pragma unroll
        for (int c = 0; c < 2 * kRuns; ++c) {
          const int at = k0 + (c >> 1) * 64 * kLowWaves + 32 * (c & 1);
          const bool in = at + 8 * q < k;
          const v4i zero = v4i{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            fx[c][i] = in ? *reinterpret_cast<const v4i*>(x[i] + at) : zero;
#pragma unroll
          for (int b = 0; b < NB; ++b)
            fd[c][b] = in ? *reinterpret_cast<const v4i*>(d[b] + at) : zero;
        }
        fence();
#pragma unroll
        for (int c = 0; c < 2 * kRuns; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[i][b] = mfma16<F16>(fd[c][b], fx[c][i], acc[i][b]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[w][i][b][lane] = acc[i][b];
      __syncthreads();
      // wave w adds block (w / NB, w % NB)
      if (w < 2 * NB) {
        const int i = w / NB, b = w % NB;
        v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kLowWaves; ++v) {
          const v4f t = sums[v][i][b][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] += t[e];
        }
        const int j = j0 + 16 * b + 4 * q;
        if ((own >> (16 * i + r) & 1) != 0 && j < rank) {
          const float f = scale[a];
          uint32_t top[4], rest[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split16<F16>(s[e] * f, top[e], rest[e]);
          uint16_t* dst = low + (row0 + 16 * i + r) * 2 * rank + j;
          *reinterpret_cast<v2i*>(dst) =
              v2i{(int)(top[0] | top[1] << 16), (int)(top[2] | top[3] << 16)};
          *reinterpret_cast<v2i*>(dst + rank) =
              v2i{(int)(rest[0] | rest[1] << 16), (int)(rest[2] | rest[3] << 16)};
        }
      }
      __syncthreads();
    }
  }
}

template <bool F16>
hipError_t launch_low(const Args& p, const uint16_t* down, const float* scale, uint16_t* low,
                      hipStream_t stream) {
  const int nb = p.r <= 16 ? 1 : p.r <= 32 ? 2 : 4;
  // as many workgroups share a block's adapters as fill the compute units
  const int64_t blocks = (p.rows_cap + kLowRows - 1) / kLowRows * ((p.r + 16 * nb - 1) / (16 * nb));
  const int64_t cap = 2 * (int64_t)device_cu_count();
  int64_t turns = cap / blocks;
  turns = turns < 1 ? 1 : turns > kLowRows ? kLowRows : turns;
  const int64_t most = p.rows_cap < p.G ? p.rows_cap : p.G;  // adapters that can meet in a block
  if (turns > most) turns = most;
  const int64_t grid = blocks * turns < cap ? blocks * turns : cap;
  const dim3 gd((unsigned)grid), bd(kLowThreads);
  const int tn = (int)turns;
  if (nb == 1)
    hipLaunchKernelGGL((lora_low_kernel<F16, 1>), gd, bd, 0, stream, p, down, scale, low, tn);
  else if (nb == 2)
    hipLaunchKernelGGL((lora_low_kernel<F16, 2>), gd, bd, 0, stream, p, down, scale, low, tn);
  else
    hipLaunchKernelGGL((lora_low_kernel<F16, 4>), gd, bd, 0, stream, p, down, scale, low, tn);
  return hipGetLastError();
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Runs the form whose tiles fit the rows a group has on average.
hipError_t launch_form(int mode, int f16, const Args& p, hipStream_t stream) {
  int64_t per = mode == kLora ? p.rows_cap : p.rows_cap / p.G;
  int64_t tiles;
  if (mode == kWgrad) {
    tiles = (int64_t)p.G * ((p.n + 255) / 256) * ((p.k + 255) / 256);
    per = 256;
  } else {
    tiles = (p.rows_cap + 255) / 256 * ((p.n + 255) / 256);
  }
  if (per >= 160 && 4 * tiles >= 3 * device_cu_count()) return launch_large(mode, f16, p, stream);
  return launch_small(mode, f16, per <= 40 ? 32 : per <= 96 ? 64 : 128, p, stream);
}

}  // namespace

size_t gemm_16bit_workspace_bytes() {
  const size_t l = large_workspace_bytes(), s = small_workspace_bytes();
  return l > s ? l : s;
}

hipError_t launch_gemm_16bit(int mode, int f16, int G, const void* a, int64_t lda, const void* b,
                             int64_t ldb, int64_t stride_b, const int64_t* offsets,
                             int64_t rows_cap, int64_t n, int64_t k, const void* c, void* out,
                             int64_t ldo, int64_t stride_o, int out_f32, void* ws, uint32_t* status,
                             hipStream_t stream) {
  Args p{};
  p.a = static_cast<const uint16_t*>(a);
  p.b = static_cast<const uint16_t*>(b);
  p.offsets = offsets;
  p.c = static_cast<const char*>(c);
  p.out = static_cast<char*>(out);
  p.lda = lda; p.ldb = ldb; p.stride_b = stride_b; p.ldo = ldo; p.stride_o = stride_o;
  p.rows_cap = rows_cap; p.n = n; p.k = k;
  p.status = status;
  p.ws = static_cast<char*>(ws);
  p.G = G; p.out_f32 = out_f32;
  return launch_form(mode, f16, p, stream);
}

size_t lora_gemm_16bit_workspace_bytes(int64_t rows_cap, int64_t n, int64_t k, int64_t r) {
  (void)n;
  (void)k;
  return gemm_16bit_workspace_bytes() + align256((size_t)rows_cap * (size_t)r * 4);
}

hipError_t launch_lora_gemm_16bit(int f16, int G, const void* x, int64_t ldx, const void* w,
                                  int64_t ldw, const void* down, const void* up,
                                  int64_t num_adapters, int64_t r, const int64_t* offsets,
                                  const int32_t* adapter, const float* scale, int64_t rows_cap,
                                  int64_t n, int64_t k, void* out, int64_t ldo, int out_f32,
                                  void* ws, uint32_t* status, hipStream_t stream) {
  if (rows_cap <= 0) return hipSuccess;
  uint16_t* low = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + gemm_16bit_workspace_bytes());
  Args p{};
  p.a = static_cast<const uint16_t*>(x);
  p.b = static_cast<const uint16_t*>(w);
  p.offsets = offsets;
  p.out = static_cast<char*>(out);
  p.lda = ldx; p.ldb = ldw; p.ldo = ldo;
  p.rows_cap = rows_cap; p.n = n; p.k = k;
  p.status = status;
  p.ws = static_cast<char*>(ws);
  p.G = G; p.out_f32 = out_f32;
  p.low = low;
  p.up = static_cast<const uint16_t*>(up);
  p.adapter = adapter;
  p.num_adapters = (int)num_adapters;
  p.r = (int)r;
  const uint16_t* d = static_cast<const uint16_t*>(down);
  const hipError_t e =
      f16 ? launch_low<true>(p, d, scale, low, stream) : launch_low<false>(p, d, scale, low, stream);
  if (e != hipSuccess) return e;
  return launch_form(kLora, f16, p, stream);
}

}  // namespace bsg
