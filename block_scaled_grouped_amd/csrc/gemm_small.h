// Grouped products, small form: 32, 64 or 128 x 128 output tiles, two
// workgroups of four wavefronts on each compute unit, every copy global -> LDS by
// the buffer unit into a ring of stages of 64 contraction indexes.
//
// For few rows the weights' bytes bound the product: a tile of 32 rows keeps two
// stages of its 16 KiB of weights in flight, two tiles a compute unit, and rows
// past the live ones are never fetched.  Contractions are split when the tiles do
// not fill the grid.
#ifndef BSG_GEMM_SMALL_H
#define BSG_GEMM_SMALL_H

#include "gemm_16bit.h"

namespace bsg {
namespace g16 {
namespace small {

constexpr int BN = 128;

// Waves of a BM x 128 tile: 2 x 2 (each BM / 2 x 64), or 1 x 4 (each 32 x 32).
template <int BM> constexpr int kWavesN = BM == 32 ? 4 : 2;
template <int BM> constexpr int kMI = BM == 128 ? 4 : 2;  // 16-row blocks
template <int BM> constexpr int kNJ = BM == 32 ? 2 : 4;   // 16-column blocks
template <int BM> constexpr int kStages = BM == 128 ? 2 : 3;  // of (BM + 128) * 128 bytes
template <int BM> constexpr int64_t kPartBytes = (int64_t)BM * BN * 4;
constexpr int kWgPerCu = 2;

template <int MODE, int BM>
struct Ring {
  static constexpr int kStageBytes = (BM + BN) * 128;
  static constexpr int kCopies = BM / 32 + BN / 32;  // per wave and stage
  Side<kColsA<MODE>, BM> a;
  Side<kColsB<MODE>, BN> b;
  uint32_t lds;
  int stages;

  // Copies stage kt into buffer s.
  __device__ __forceinline__ void copy(int kt, int s) const {
    const bool live = kt < stages;
    const uint32_t at = lds + s * kStageBytes;
    const v4i ra = a.rsrc(kt, live), rb = b.rsrc(kt, live);
    const uint64_t ma = a.mask(kt, stages), mb = b.mask(kt, stages);
    static_for<BM / 32>([&](auto i) {
      constexpr int I = decltype(i)::value;
      a.template copy<I, I * 4096>(ra, at, ma);
    });
    static_for<BN / 32>([&](auto i) {
      constexpr int I = decltype(i)::value;
      b.template copy<I, BM * 128 + I * 4096>(rb, at, mb);
    });
  }
};

template <int MODE, bool F16, int BM>
__device__ __forceinline__ void contract(uint32_t lds, const Tile& t, int w, int lane,
                                         v4f (&acc)[kMI<BM>][kNJ<BM>]) {
  constexpr int MI = kMI<BM>, NJ = kNJ<BM>, NS = kStages<BM>;
  Ring<MODE, BM> ring;
  ring.stages = uni((t.kl + kStageK - 1) / kStageK);
  if (ring.stages == 0) return;
  ring.a.init(t.a, t.lda, t.a_rows, t.kl, w, lane);
  ring.b.init(t.b, t.ldb, t.b_rows, t.kl, w, lane);
  ring.lds = uni(lds + w * 1024);
  FragOff<kColsA<MODE>, BM, MI> fa;
  FragOff<kColsB<MODE>, BN, NJ> fb;
  fa.init(lds, (w / kWavesN<BM>) * (16 * MI), lane);
  fb.init(lds + BM * 128, (w % kWavesN<BM>) * (16 * NJ), lane);
  static_for<NS - 1>([&](auto s) { ring.copy(decltype(s)::value, decltype(s)::value); });
  int s = 0;
  for (int kt = 0; kt < ring.stages; ++kt) {
    // stage kt has landed for every wave, and every wave has read stage kt - 1,
    // whose buffer takes the next copies
    wait_and_barrier<(NS - 2) * Ring<MODE, BM>::kCopies>();
    const int next = s == 0 ? NS - 1 : s - 1;
    ring.copy(kt + NS - 1, next);
    const uint32_t at = s * Ring<MODE, BM>::kStageBytes;
    static_for<2>([&](auto tc) {
      constexpr int T = decltype(tc)::value;
      v4i a[MI], b[NJ];
      static_for<MI>([&](auto i) {
        a[decltype(i)::value] = fa.template read<decltype(i)::value, T>(at);
      });
      static_for<NJ>([&](auto j) {
        b[decltype(j)::value] = fb.template read<decltype(j)::value, T>(at);
      });
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma_step<MODE, F16>(b[j], a[i], acc[i][j]);
    });
    s = s + 1 == NS ? 0 : s + 1;
  }
}

template <int MODE, bool F16, int BM>
__global__ __launch_bounds__(kThreads, kWgPerCu) void small_kernel(Args p) {
  constexpr int MI = kMI<BM>, NJ = kNJ<BM>;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kStages<BM> * (BM + BN) * 128];
  __shared__ Sched sm;
  __shared__ int ids[MODE == kLora ? BM : 1];
  const uint32_t lds = lds_offset(ring);
  const int total = count_tiles<MODE, BM, BN>(p, sm);
  const Rounds rounds = plan_rounds<MODE, true>(p, total);
  const int nsplit = rounds.nsplit;
  for (int round = 0;; ++round) {
    const Work work = take_work(p, rounds, round);
    if (work.tile < 0) break;
    Tile t = find_tile<MODE, BM, BN>(p, sm, uni(work.tile));
    if (work.part >= 0) narrow_tile<MODE>(t, uni(work.part), nsplit);
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, w = uni(tid >> 6);
    const int wrow = (w / kWavesN<BM>) * (16 * MI), wcol = (w % kWavesN<BM>) * (16 * NJ);
    v4f acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (MODE == kLora) tile_adapters<BM>(p, sm, t, ids);
    contract<MODE, F16, BM>(lds, t, w, lane, acc);
    // every copy has landed and no wave still reads the ring before the next
    // tile's first copies
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if constexpr (MODE == kLora) {
      add_low_rank<F16, MI, NJ>(p, t, ids, wrow, wcol, lane, uni(work.part), work.nparts, acc);
      __syncthreads();  // ids are read before the next tile's
    }
    if (work.part >= 0) {
      write_split_record<MODE>(p.ws, work.slot, nsplit, t);
      store_part<MI, NJ>(
          reinterpret_cast<float*>(p.ws + kWsHeader + (int64_t)work.slot * kPartBytes<BM>), acc, w, lane,
          wrow, t.a_rows);
    } else {
      store_blocks<MODE, F16, MI, NJ>(acc, out_tile<MODE>(p, t), p.out_f32, wrow, wcol, lane);
    }
  }
}

template <int MODE, bool F16, int BM>
hipError_t launch(Args p, hipStream_t stream) {
  const int grid = prepare_launch<MODE, BM, BN>(p, kWgPerCu * device_cu_count());
  if (grid == 0) return hipSuccess;
  hipLaunchKernelGGL((small_kernel<MODE, F16, BM>), dim3(grid), dim3(kThreads), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.ws == nullptr) return e;
  hipLaunchKernelGGL((split_reduce_kernel<MODE == kInt8, F16, BM, BN, kWavesN<BM>, kMI<BM>, kNJ<BM>>),
                     dim3(reduce_grid(grid, BM * BN / 512)), dim3(kThreads), 0, stream, p.ws, p.out,
                     p.c, p.ldo, p.out_f32, p.a_scales, p.b_scales);
  return hipGetLastError();
}

}  // namespace small
}  // namespace g16
}  // namespace bsg

#endif  // BSG_GEMM_SMALL_H
