// 16-bit grouped products, large form: 256 x 256 output tiles, one persistent
// workgroup of four wavefronts on each compute unit, each wave 128 x 128 of the
// output as 4 x 4 blocks of 32 x 32 (256 accumulator registers a lane).
//
// A stage is 64 contraction indexes (32 KiB an operand); two LDS buffers.  While
// stage s is consumed from one, stage s + 1 lands in the other, and the copies of
// stage s + 2 are issued as soon as stage s's last fragments are in registers.
// A goes global -> LDS by the buffer unit, B through registers (loads issued a
// stage ahead, written to LDS half a stage later): the direct path alone does not
// feed a compute unit at the rate its matrix units consume.  The schedule of each
// half stage is written out instruction by instruction and fenced, so that the
// compiler keeps it; one barrier a stage.
#include "gemm_16bit.h"

namespace bsg {
namespace g16 {

namespace {

constexpr int BM = 256, BN = 256;
constexpr int kTileBytes = 256 * 128;
constexpr int kBufBytes = 2 * kTileBytes;
constexpr int kPieces = 8;          // per wave, operand and stage
constexpr int kBarrierSlot = 4;     // matrix instruction of a stage's second half that
                                    // the barrier follows
constexpr int64_t kPartBytes = (int64_t)BM * BN * 4;

typedef v4i Half[2][4];  // fragments of 32 contraction indexes: [k16 step][block]

template <int MODE>
struct Copies {
  Side<kColsA<MODE>, BM> a;
  Side<kColsB<MODE>, BN> b;
  int bslot;  // this lane's LDS offset of a piece of B
  uint32_t lds;
  int w;
};

__device__ __forceinline__ uint32_t buf_a(uint32_t lds, int s) { return lds + s * kBufBytes; }
__device__ __forceinline__ uint32_t buf_b(uint32_t lds, int s) {
  return lds + s * kBufBytes + kTileBytes;
}

template <int P, int MODE>
__device__ __forceinline__ void copy_a(const Copies<MODE>& c, v4i rsrc, int s, int kt) {
  dma16(rsrc, buf_a(c.lds, s) + c.w * 1024 + P * 4096, c.a.piece_off(P, kt));
}

template <int Q, int MODE>
__device__ __forceinline__ void load_b(const Copies<MODE>& c, __amdgpu_buffer_rsrc_t rsrc, int kt,
                                       v4i (&stage)[kPieces]) {
  stage[Q] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, c.b.piece_off(Q, kt), 0, 0);
}

template <int Q, int MODE>
__device__ __forceinline__ void store_b(const Copies<MODE>& c, int s, const v4i (&stage)[kPieces]) {
  *reinterpret_cast<lds_v4i*>((size_t)(buf_b(c.lds, s) + c.bslot + Q * 4096)) = stage[Q];
}

template <int MODE>
__device__ __forceinline__ v4i a_rsrc(const Copies<MODE>& c, int kt, int stages) {
  return rsrc_words(c.a.stage_base(kt), c.a.stage_range(kt, kt < stages));
}
template <int MODE>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t b_rsrc(const Copies<MODE>& c, int kt, int stages) {
  return make_rsrc(reinterpret_cast<const void*>(c.b.stage_base(kt)),
                   c.b.stage_range(kt, kt < stages));
}

// Fragment Q of the 16 of half S of a stage, in the order the matrix instructions
// first use them: for each k16 step A0, B0, B1, B2, B3, A1, A2, A3.
template <int MODE, int S, int Q>
__device__ __forceinline__ void read_frag(uint32_t lds, int s,
                                          const FragOff<kColsA<MODE>, BM, 4>& fa,
                                          const FragOff<kColsB<MODE>, BN, 4>& fb, Half& a, Half& b) {
  constexpr int u = Q >> 3, k = Q & 7, T = 2 * S + u;
  if constexpr (k == 0 || k >= 5) {
    constexpr int i = k == 0 ? 0 : k - 4;
    a[u][i] = fa.template read<i, T>(buf_a(lds, s));
  } else {
    b[u][k - 1] = fb.template read<k - 1, T>(buf_b(lds, s));
  }
}

template <bool F16, int M>
__device__ __forceinline__ void mfma(const Half& a, const Half& b, v16f (&acc)[4][4]) {
  constexpr int u = M >> 4, i = (M >> 2) & 3, j = M & 3;
  acc[i][j] = mfma16<F16>(b[u][j], a[u][i], acc[i][j]);
  // the intrinsic has no side effects, so passes may sink it past the fences; an
  // opaque use of its result keeps it in place
  asm volatile("" : "+a"(acc[i][j]));
}

// One tile's contraction.
template <int MODE, bool F16>
__device__ __forceinline__ void contract(uint32_t lds, const Tile& t, int w, int lane,
                                         v16f (&acc)[4][4]) {
  const int stages = uni((t.kl + kStageK - 1) / kStageK);
  if (stages == 0) return;
  Copies<MODE> c;
  c.a.init(t.a, t.lda, t.a_rows, t.kl, w, lane, false);
  c.b.init(t.b, t.ldb, t.b_rows, t.kl, w, lane, true);
  c.bslot = Side<kColsB<MODE>, BN>::slot(w, lane);
  c.lds = lds;
  c.w = w;
  FragOff<kColsA<MODE>, BM, 4> fa;
  FragOff<kColsB<MODE>, BN, 4> fb;
  fa.init((w >> 1) * 128, lane);
  fb.init((w & 1) * 128, lane);

  // stage 0 into buffer 0; stage 1's A into buffer 1 and its B into registers
  v4i stage[kPieces];
  {
    const __amdgpu_buffer_rsrc_t r = b_rsrc(c, 0, stages);
    static_for<kPieces>([&](auto q) { load_b<decltype(q)::value>(c, r, 0, stage); });
    const v4i ra = a_rsrc(c, 0, stages);
    static_for<kPieces>([&](auto q) { copy_a<decltype(q)::value>(c, ra, 0, 0); });
    static_for<kPieces>([&](auto q) { store_b<decltype(q)::value>(c, 0, stage); });
    const v4i ra1 = a_rsrc(c, 1, stages);
    static_for<kPieces>([&](auto q) { copy_a<decltype(q)::value>(c, ra1, 1, 1); });
    const __amdgpu_buffer_rsrc_t r1 = b_rsrc(c, 1, stages);
    static_for<kPieces>([&](auto q) { load_b<decltype(q)::value>(c, r1, 1, stage); });
  }
  wait_and_barrier<2 * kPieces>();
  Half a0, b0, a1, b1;
  static_for<16>([&](auto q) { read_frag<MODE, 0, decltype(q)::value>(lds, 0, fa, fb, a0, b0); });
  for (int kt = 0; kt < stages; ++kt) {
    const int s = kt & 1;
    const __amdgpu_buffer_rsrc_t rb = b_rsrc(c, kt + 2, stages);
    const v4i ra = a_rsrc(c, kt + 2, stages);
    // first half: the second half's fragments (same buffer), then, one register at
    // a time, stage kt + 1's B into the other buffer and the loads of stage kt + 2's
    static_for<32>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      mfma<F16, m>(a0, b0, acc);
      fence();
      if constexpr (m < 16) {
        read_frag<MODE, 1, m>(lds, s, fa, fb, a1, b1);
      } else if constexpr (m % 2 == 0) {
        constexpr int q = (m - 16) / 2;
        store_b<q>(c, s ^ 1, stage);
        load_b<q>(c, rb, kt + 2, stage);
      }
      fence();
    });
    // second half: after the barrier the other buffer holds stage kt + 1 for every
    // wave and this one is free: A of stage kt + 2 into it, and the first fragments
    // of stage kt + 1
    static_for<32>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      mfma<F16, m>(a1, b1, acc);
      fence();
      if constexpr (m == kBarrierSlot) wait_and_barrier<kPieces>();
      if constexpr (m >= kBarrierSlot) {
        constexpr int q = m - kBarrierSlot;
        if constexpr (q < 16) read_frag<MODE, 0, q>(lds, s ^ 1, fa, fb, a0, b0);
        if constexpr (q % 3 == 1 && q / 3 < kPieces) copy_a<q / 3>(c, ra, s, kt + 2);
      }
      fence();
    });
  }
}

template <int MODE, bool F16>
__global__ __launch_bounds__(kThreads) void large_kernel(Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * kBufBytes];
  __shared__ Sched sm;
  __shared__ int ids[MODE == kLora ? BM : 1];
  const uint32_t lds = lds_offset(ring);
  const int total = count_tiles<MODE, BM, BN>(p, sm);
  const int grid = (int)gridDim.x, left = total % grid;
  const int nsplit =
      p.ws == nullptr
          ? 1
          : split_parts(grid, left,
                        (int)(((MODE == kWgrad ? p.rows_cap : p.k) + kStageK - 1) / kStageK), 4);
  write_split_header(p.ws, total, nsplit);
  const int slot = xcd_slot();
  for (int round = 0;; ++round) {
    const Work work = take_work(round, slot, total, nsplit);
    if (work.tile < 0) break;
    Tile t = find_tile<MODE, BM, BN>(p, sm, uni(work.tile));
    if (work.part >= 0) narrow_tile<MODE>(t, uni(work.part), nsplit);
    // opaque per-tile copy of the thread index: keeps the offsets of the tile body
    // from being hoisted out of the persistent loop
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, w = uni(tid >> 6);
    const int wrow = (w >> 1) * 128, wcol = (w & 1) * 128;
    v16f acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = v16f{};
    if constexpr (MODE == kLora) tile_adapters<BM>(p, sm, t, ids);
    contract<MODE, F16>(lds, t, w, lane, acc);
    // every copy has landed and no wave still reads a buffer before the next
    // tile's first copies
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if constexpr (MODE == kLora) {
      add_low_rank<F16, 4, 4>(p, t, ids, wrow, wcol, lane, uni(work.part), work.nparts, acc);
      __syncthreads();  // ids are read before the next tile's
    }
    if (work.part >= 0) {
      write_split_record(p.ws, slot, nsplit, t);
      store_part<4, 4>(reinterpret_cast<float*>(p.ws + kWsHeader + (int64_t)slot * kPartBytes), acc,
                       w, lane, wrow, t.a_rows);
    } else {
      store_blocks<F16, 4, 4>(acc, out_tile(p, t), p.out_f32, wrow, wcol, lane);
    }
  }
}

template <int MODE, bool F16>
hipError_t launch(const Args& p, hipStream_t stream) {
  int64_t bound;
  if (MODE == kWgrad) bound = (int64_t)p.G * ((p.n + BM - 1) / BM) * ((p.k + BN - 1) / BN);
  else bound = ((p.rows_cap + BM - 1) / BM + (MODE == kLora ? 0 : p.G)) * ((p.n + BN - 1) / BN);
  const int cus = device_cu_count();
  const int64_t kl = MODE == kWgrad ? p.rows_cap : p.k;
  const int parts = p.ws != nullptr ? split_parts(cus, 1, (int)((kl + kStageK - 1) / kStageK), 4) : 1;
  int64_t grid = bound * parts < cus ? bound * parts : cus;
  if (grid <= 0) return hipSuccess;
  hipLaunchKernelGGL((large_kernel<MODE, F16>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts < 2) return e;
  hipLaunchKernelGGL((split_reduce_kernel<F16, BM, BN, 2, 4, 4>), dim3((unsigned)cus),
                     dim3(kThreads), 0, stream, p.ws, p.out, p.c, p.ldo, p.out_f32);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_mode(int mode, const Args& p, hipStream_t stream) {
  if (mode == kFprop) return launch<kFprop, F16>(p, stream);
  if (mode == kWgrad) return launch<kWgrad, F16>(p, stream);
  if (mode == kDgrad) return launch<kDgrad, F16>(p, stream);
  return launch<kLora, F16>(p, stream);
}

}  // namespace

hipError_t launch_large(int mode, int f16, const Args& p, hipStream_t stream) {
  return f16 ? launch_mode<true>(mode, p, stream) : launch_mode<false>(mode, p, stream);
}

size_t large_workspace_bytes() {
  return (size_t)kWsHeader + (size_t)device_cu_count() * (size_t)kPartBytes;
}

}  // namespace g16
}  // namespace bsg
