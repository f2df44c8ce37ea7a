// 16-bit grouped products: which form runs, and the first product of the adapters.
#include "gemm_16bit.h"

namespace bsg {

using namespace g16;

namespace {

// The adapters' first product, X[t, :] A_a^T: as 16-bit values, or (parts of the
// contraction) as it is.
//
// A workgroup of eight waves takes 32 consecutive rows, 16 NB rank columns, one of
// the adapters that occur in those rows and one part of the contraction; the waves
// take turns at the part's runs of 64 (a 128-byte line of a row) and their sums are
// added through LDS in one order.  Rows of another adapter are neither read nor
// written.  Operands come straight from memory: nothing is shared between waves
// that LDS could serve.  A compute unit takes 64 GB/s that way, 28 past its L2, so
// where the rows are few, 16 rank columns and a part of the contraction make a
// workgroup, and the second product adds the parts.
constexpr int kLowThreads = 512;
constexpr int kLowWaves = kLowThreads / 64;
constexpr int kLowRows = 32;
constexpr int64_t kFewRows = 1024;  // 32 blocks of rows leave compute units idle

// NB: 16 NB <= 64 rank columns a workgroup.  DENSE: two workgroups a compute unit, with fewer
// loads in flight in each.  For all calls of 16 columns, and for few rows, where most
// workgroups are later turns that have nothing to do (660 rows, rank 32, 25 adapters of fp16:
// the call in 13.2 us, 15.2 with one workgroup a compute unit).
template <bool F16, int NB, bool DENSE>
__global__ __launch_bounds__(kLowThreads, DENSE ? 4 : 2) void lora_low_kernel(Args p, const uint16_t* down,
                                                               int turns) {
  __shared__ int64_t off[kMaxGroups + 1];
  __shared__ int adapters[kMaxGroups];
  __shared__ __attribute__((aligned(16))) v4f sums[kLowWaves][2][NB][64];
  __shared__ float peaks[2][NB][16];  // largest magnitudes of a row's 16 columns
  for (int g = threadIdx.x; g < p.G; g += kLowThreads) {
    adapters[g] = adapter_of(p, g);
    if (blockIdx.x == 0 && p.adapter[g] >= p.num_adapters) dev_status_or(p.status, kDevBadAdapter);
  }
  load_offsets_clamped(p.offsets, p.G, p.rows_cap, off, nullptr);
  __syncthreads();
  const int64_t first = uni64(off[0]), last = uni64(off[p.G]);
  const int lane = threadIdx.x & 63, w = uni((int)(threadIdx.x >> 6));
  const int r = lane & 15, q = lane >> 4, rank = p.r, k = (int)p.k;
  const int rank_blocks = (rank + 16 * NB - 1) / (16 * NB);
  const int parts = p.low_parts;
  uint16_t* low16 = static_cast<uint16_t*>(p.low);
  float* low32 = static_cast<float*>(p.low);
  const int chunks = (rank + kLowChunk - 1) / kLowChunk;
  const int64_t blocks = (last - first + kLowRows - 1) / kLowRows * rank_blocks;
  const int64_t items = blocks * turns * parts;
  const int runs = (k + 63) / 64;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    // the turns come last: most blocks hold one adapter, and their later turns nothing
    const int part = uni((int)(item % parts));
    const int64_t it = item / parts % blocks;
    const int run0 = runs * part / parts, run1 = runs * (part + 1) / parts;
    const int turn0 = uni((int)(item / parts / blocks));
    const int j0 = uni((int)(it % rank_blocks)) * (16 * NB);
    const int64_t row0 = first + it / rank_blocks * kLowRows;
    // lane l: adapter of row l % 32
    const int64_t mine_row = row0 + (lane & 31);
    const int id = mine_row < last ? adapters[request_of(off, p.G, mine_row)] : -1;
    // rows past the last, rank columns past the last and chunks past the contraction
    // read as zeros
    const int ldx2 = (int)(p.lda * 2), k2 = k * 2;
    const int64_t rows = last - row0;
    const __amdgpu_buffer_rsrc_t x =
        make_rsrc(p.a + row0 * p.lda, (rows < kLowRows ? rows : kLowRows) * ldx2);
    uint32_t todo = (uint32_t)__ballot(id >= 0);
    int turn = 0;
    while (todo != 0) {
      const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
      const uint32_t own = (uint32_t)__ballot(id == a);
      todo &= ~own;
      const bool mine = turn == turn0;
      turn = turn + 1 == turns ? 0 : turn + 1;
      if (!mine) continue;
      const int left = rank - j0;
      const __amdgpu_buffer_rsrc_t d = make_rsrc(down + ((int64_t)a * rank + j0) * p.k,
                                                 (int64_t)(left < 16 * NB ? left : 16 * NB) * k2);
      v4f acc[2][NB];
      uint32_t xrow[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xrow[i] = (own >> (16 * i + r) & 1) != 0 ? (uint32_t)((16 * i + r) * ldx2)
                                                 : (uint32_t)kDmaOutOfRange;
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[i][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      }
      // kRuns of the wave's runs are loaded before the first is used
      constexpr int kRuns = DENSE ? (NB == 1 ? 3 : NB == 2 ? 2 : 1) : NB == 2 ? 4 : 2;
      const int end = 64 * run1 < k ? 64 * run1 : k;
      for (int k0 = 64 * (run0 + w); k0 < end; k0 += 64 * kLowWaves * kRuns) {
        v4i fx[2 * kRuns][2], fd[2 * kRuns][NB];
#pragma unroll
        for (int c = 0; c < 2 * kRuns; ++c) {
          const int at = k0 + (c >> 1) * 64 * kLowWaves + 32 * (c & 1);
          const uint32_t o = at + 8 * q < end ? 2 * (at + 8 * q) : kDmaOutOfRange;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            fx[c][i] = __builtin_amdgcn_raw_buffer_load_b128(x, (int)(o + xrow[i]), 0, 0);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            fd[c][b] = __builtin_amdgcn_raw_buffer_load_b128(d, (int)(o + (16 * b + r) * k2), 0, 0);
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
      const int i = w / NB % 2, b = w % NB;
      v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (w < 2 * NB) {
#pragma unroll
        for (int v = 0; v < kLowWaves; ++v) {
          const v4f t = sums[v][i][b][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] += t[e];
        }
      }
      LowScales f{1.0f, 1.0f};
      if constexpr (F16) {
        if (parts == 1) {
          float m = fmaxf(fmaxf(fabsf(s[0]), fabsf(s[1])), fmaxf(fabsf(s[2]), fabsf(s[3])));
          m = fmaxf(m, __shfl_xor(m, 16, 64));
          m = fmaxf(m, __shfl_xor(m, 32, 64));
          if (w < 2 * NB && q == 0) peaks[i][b][r] = m;
          __syncthreads();
#pragma unroll
          for (int c = 0; c < NB; ++c) m = fmaxf(m, peaks[i][c][r]);
          f = low_scales(m);
        }
      }
      const int j = j0 + 16 * b + 4 * q;
      const int64_t row = row0 + 16 * i + r;
      if (w < 2 * NB && (own >> (16 * i + r) & 1) != 0 && j < rank) {
        if (parts > 1) {
          float* dst = low32 + (part * p.rows_cap + row) * rank + j;
          *reinterpret_cast<v4f*>(dst) = s;
        } else {
          uint32_t lo[kLowValues], hi[kLowValues];
          split_low<F16>(s[0] * f.down, s[1] * f.down, lo);
          split_low<F16>(s[2] * f.down, s[3] * f.down, hi);
          uint16_t* dst = low16 + row * kLowValues * rank + j;
#pragma unroll
          for (int h = 0; h < kLowValues; ++h)
            *reinterpret_cast<v2i*>(dst + h * rank) = v2i{(int)lo[h], (int)hi[h]};
          if (F16 && b == 0 && q == 0) p.low_power[row * chunks + j0 / kLowChunk] = f.up;
        }
      }
      __syncthreads();
    }
  }
}

// Parts of the first product's contraction: several where the rows are few.
int low_parts(int64_t rows_cap, int64_t k) {
  return rows_cap <= kFewRows && k >= 1024 ? kLowParts : 1;
}

template <bool F16>
hipError_t launch_low(const Args& p, const uint16_t* down, hipStream_t stream) {
  // the rank columns that share a power of two (fp16, where no parts are left to the second
  // product) are a workgroup's
  static_assert(kLowChunk == 64, "16 * 4 columns");
  const bool few = p.rows_cap <= kFewRows;
  const bool narrow = p.r <= 16 || (few && (!F16 || p.low_parts > 1));
  const int nb = narrow ? 1 : p.r <= 32 ? 2 : 4;
  // as many workgroups share a block's adapters as fill the compute units
  const int64_t blocks = (p.rows_cap + kLowRows - 1) / kLowRows *
                         ((p.r + 16 * nb - 1) / (16 * nb)) * p.low_parts;
  const int64_t cap = 2 * (int64_t)device_cu_count();
  int64_t turns = cap / blocks;
  turns = turns < 1 ? 1 : turns > kLowRows ? kLowRows : turns;
  const int64_t most = p.rows_cap < p.G ? p.rows_cap : p.G;  // adapters that can meet in a block
  if (turns > most) turns = most;
  const int64_t grid = blocks * turns < cap ? blocks * turns : cap;
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kLowThreads), 0, stream, p, down,
                       (int)turns);
  };
  bool done = nb == 1;
  if (done) run(lora_low_kernel<F16, 1, true>);
  if constexpr (F16) {
    if (!done && few) {
      if (nb == 2) run(lora_low_kernel<F16, 2, true>);
      else run(lora_low_kernel<F16, 4, true>);
      done = true;
    }
  }
  if (!done) {
    if (nb == 2) run(lora_low_kernel<F16, 2, false>);
    else run(lora_low_kernel<F16, 4, false>);
  }
  return hipGetLastError();
}

// Bytes a row of what the first product leaves for the second.
size_t low_values_bytes(int64_t r) { return (size_t)(2 * kLowValues * r); }
size_t low_power_bytes(int64_t r) { return (size_t)(4 * ((r + kLowChunk - 1) / kLowChunk)); }

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// The form with the least expected time, by what a round of tiles costs in each:
//   stages of the longest workgroup * us a stage + us a tile + us of the second step
// where the last round is split.  Measured with every slot taken: a stage of 64
// contraction indexes costs a workgroup 1.37 us with 256 x 256 tiles (1.57 PFLOP/s in
// all), 1.14, 0.70 and 0.52 us with 128, 64 and 32 x 128 (0.94, 0.77 and 0.52
// PFLOP/s, two workgroups a compute unit).  So large tiles win where they fill the
// chip, and small ones where few rows, short contractions or narrow outputs leave
// them idle: 16384 x 14336 x 4096 in 8 groups 1.39 against 2.05 ms (128) and 3.72 ms
// (32), 844 rows of three groups x 312 x 2864 31 (256) against 23 us (64).  Over 170
// calls of random sizes the choice costs 1 % over the best of the four.  Group sizes
// are on the device, so a nonempty group counts for half a tile more than its rows.
struct Form {
  int bm, bn;
  double stage_us, tile_us, reduce_us;
};
constexpr Form kForms[4] = {
    {32, 128, 0.52, 1.5, 4.0}, {64, 128, 0.70, 2.0, 4.5}, {128, 128, 1.14, 3.0, 6.0},
    {256, 256, 1.37, 5.0, 13.0}};

double expected_us(const Form& f, int mode, int64_t G, int64_t rows_cap, int64_t n, int64_t k,
                   bool split) {
  const int64_t slots = (f.bm == 256 ? 1 : 2) * (int64_t)device_cu_count();
  const int64_t ntn = (n + f.bn - 1) / f.bn;
  int64_t tiles, stages, split_stages;
  if (mode == kWgrad) {
    tiles = G * ((n + f.bm - 1) / f.bm) * ((k + f.bn - 1) / f.bn);
    split_stages = (rows_cap + kStageK - 1) / kStageK;
    stages = (rows_cap / G + kStageK - 1) / kStageK;
    if (stages < 1) stages = 1;
  } else {
    const int64_t groups = mode == kLora ? 1 : rows_cap < G ? rows_cap : G;
    tiles = ((rows_cap + f.bm - 1) / f.bm + (groups > 1 ? groups / 2 : 0)) * ntn;
    split_stages = stages = (k + kStageK - 1) / kStageK;
  }
  const int64_t full = tiles / slots, left = tiles % slots;
  double us = (double)full * ((double)stages * f.stage_us + f.tile_us);
  if (left > 0) {
    const int parts = split ? split_parts((int)slots, (int)left, (int)split_stages) : 1;
    us += (double)((stages + parts - 1) / parts) * f.stage_us + f.tile_us +
          (parts > 1 ? f.reduce_us : 0.0);
  }
  return us;
}

hipError_t launch_form(int mode, int f16, const Args& p, hipStream_t stream) {
  const int bm = form_rows(mode, p.G, p.rows_cap, p.n, p.k, p.ws != nullptr);
  return bm == 256 ? launch_large(mode, f16, p, stream) : launch_small(mode, f16, bm, p, stream);
}

}  // namespace

namespace g16 {

// Rows of the tiles of the form that a call takes.
int form_rows(int mode, int64_t G, int64_t rows_cap, int64_t n, int64_t k, bool split) {
  int best = mode == kWgrad ? 2 : 0;  // weight gradients have no forms of fewer rows
  double us = expected_us(kForms[best], mode, G, rows_cap, n, k, split);
  for (int i = best + 1; i < 4; ++i) {
    const double t = expected_us(kForms[i], mode, G, rows_cap, n, k, split);
    if (t < us) {
      us = t;
      best = i;
    }
  }
  return kForms[best].bm;
}

}  // namespace g16

size_t gemm_16bit_workspace_bytes() {
  const size_t l = large_workspace_bytes(), s = small_workspace_bytes();
  return l > s ? l : s;
}

int gemm_16bit_tile_rows(int mode, int64_t G, int64_t rows_cap, int64_t n, int64_t k, bool split) {
  return form_rows(mode, G, rows_cap, n, k, split);
}

int lora_gemm_16bit_tile_rows(int64_t rows_cap, int64_t n, int64_t k) {
  return form_rows(kLora, 1, rows_cap, n, k, true);
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

// Never less for more rows or a larger rank, and the same for every n and k, so that the
// workspace of the largest call serves all: the parts of few rows take more than the values
// of a few rows more.
size_t lora_gemm_16bit_workspace_bytes(int64_t rows_cap, int64_t r) {
  const size_t few = (size_t)(rows_cap < kFewRows ? rows_cap : kFewRows);
  const size_t parts = few * (size_t)r * 4 * kLowParts;
  const size_t values = (size_t)rows_cap * (low_values_bytes(r) + low_power_bytes(r));
  return gemm_16bit_workspace_bytes() + align256(parts > values ? parts : values);
}

hipError_t launch_lora_gemm_16bit(int f16, int G, const void* x, int64_t ldx, const void* w,
                                  int64_t ldw, const void* down, const void* up,
                                  int64_t num_adapters, int64_t r, const int64_t* offsets,
                                  const int32_t* adapter, const float* scale, int64_t rows_cap,
                                  int64_t n, int64_t k, void* out, int64_t ldo, int out_f32,
                                  void* ws, uint32_t* status, hipStream_t stream) {
  if (rows_cap <= 0) return hipSuccess;
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
  p.low = static_cast<char*>(ws) + gemm_16bit_workspace_bytes();
  p.low_parts = low_parts(rows_cap, k);
  p.low_power =
      reinterpret_cast<float*>(static_cast<char*>(p.low) + (size_t)rows_cap * low_values_bytes(r));
  p.scale = scale;
  p.up = static_cast<const uint16_t*>(up);
  p.adapter = adapter;
  p.num_adapters = (int)num_adapters;
  p.r = (int)r;
  const uint16_t* d = static_cast<const uint16_t*>(down);
  const hipError_t e = f16 ? launch_low<true>(p, d, stream) : launch_low<false>(p, d, stream);
  if (e != hipSuccess) return e;
  return launch_form(kLora, f16, p, stream);
}

}  // namespace bsg
