// Grouped products, large form: 256 x 256 output tiles, one persistent
// workgroup of four wavefronts on each compute unit, each wave 128 x 128 of the
// output as 8 x 8 blocks of 16 x 16 (256 accumulator registers a lane).
//
// A stage is 64 contraction indexes (32 KiB an operand); two LDS buffers.  While
// stage s is consumed from one, stage s + 1 lands in the other, and the copies of
// stage s + 2 go into a buffer as soon as every wave has its last fragments in
// registers.  All copies go global -> LDS by the buffer unit.  The schedule of a
// stage is written out, instruction by instruction, and fenced, so that the compiler
// keeps it: a matrix instruction takes 16 cycles, in which a wave can issue three
// others, and what is issued in excess of that idles the matrix unit (one wave is
// all that a SIMD holds beside 256 accumulators).
//
// What bounds it: power, with random operands, and what is left of a stage's issue:
// 2251 cycles a stage of 2048 at 16384 x 14336 x 4096 (with copies four instructions
// apart and each begun and ended in one slot 2434, six apart 2374; without copies
// 2115).  1.50 PFLOP/s there, 1.54 at 16384 x 4096 x 14336, in any of the three
// modes 1.45 or more (library: 1.55, 1.34 and 1.13 for FPROP, DGRAD and WGRAD).
#ifndef BSG_GEMM_LARGE_H
#define BSG_GEMM_LARGE_H

#include "gemm_16bit.h"

namespace bsg {
namespace g16 {
namespace large {

constexpr int BM = 256, BN = 256;
constexpr int kTileBytes = 256 * 128;
constexpr int kBufBytes = 2 * kTileBytes;  // A's tile, then B's
// Places in a stage's 128 matrix instructions: where its buffer is free for the
// next copies, where the next stage has to be there, and the copies between (the
// last is issued 97 of them before its stage has to be there).
constexpr int kFreeSlot = 36;
constexpr int kReadySlot = 96;
constexpr int kCopySlot = 37, kCopyStep = 6;
constexpr int kCopies = 16;  // per wave and stage: 8 of A, 8 of B
constexpr int kCopiesBeforeReady = (kReadySlot - kCopySlot + kCopyStep - 1) / kCopyStep;
static_assert(kCopySlot + (kCopies - 1) * kCopyStep < 128 && kReadySlot + 32 <= 128 &&
                  kReadySlot - kFreeSlot >= 34,
              "schedule");
constexpr int64_t kPartBytes = (int64_t)BM * BN * 4;

typedef v4i Half[8];  // an operand's fragments of 32 contraction indexes

// This wave's copies of a stage.
template <int MODE>
struct Copies {
  Side<kColsA<MODE>, BM> a;
  Side<kColsB<MODE>, BN> b;
  uint32_t lds;   // of the buffer that is being copied to
  int stages;
  v4i ra, rb;     // descriptors and lanes of the stage that is being copied
  uint64_t ma, mb;

  __device__ __forceinline__ void begin(int kt) {
    const bool live = kt < stages;
    ra = a.rsrc(kt, live);
    rb = b.rsrc(kt, live);
    ma = a.mask(kt, stages);
    mb = b.mask(kt, stages);
  }
  template <int P>
  __device__ __forceinline__ int copy_begin() const {
    if constexpr (P < 8) return a.template copy_begin<P, P * 4096>(lds, ma);
    else return b.template copy_begin<P - 8, kTileBytes + (P - 8) * 4096>(lds, mb);
  }
  template <int P>
  __device__ __forceinline__ void copy_end(int off) const {
    copy16_end(P < 8 ? ra : rb, off);
  }
};

// Fragment Q of the 16 of half S of a stage, in the order the matrix instructions
// first use them: A0, B0 .. B7, A1 .. A7.
template <int MODE, int S, int Q>
__device__ __forceinline__ void read_frag(const FragOff<kColsA<MODE>, BM, 8>& fa,
                                          const FragOff<kColsB<MODE>, BN, 8>& fb, Half& a, Half& b) {
  if constexpr (Q == 0 || Q >= 9) {
    constexpr int i = Q == 0 ? 0 : Q - 8;
    a[i] = fa.template read<i, S>();
  } else {
    b[Q - 1] = fb.template read<Q - 1, S>();
  }
}

// The instruction itself, its accumulator tied to its own registers: left to
// the intrinsic, the register allocator moves a good part of the 256 accumulators
// around in every stage.  Its operands come from LDS reads (for whose arrival the
// compiler waits), never from a vector instruction right before it, and an
// accumulator is used again 64 instructions later, so it needs no wait states here;
// mfma_drain() ends a run of them.
template <int MODE, bool F16, int M>
__device__ __forceinline__ void mfma(const Half& a, const Half& b, v4f (&acc)[8][8]) {
  if constexpr (MODE == kInt8)
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0"
                 : "+a"(acc[M >> 3][M & 7])
                 : "v"(b[M & 7]), "v"(a[M >> 3]));
  else if constexpr (F16)
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0"
                 : "+a"(acc[M >> 3][M & 7])
                 : "v"(b[M & 7]), "v"(a[M >> 3]));
  else
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
                 : "+a"(acc[M >> 3][M & 7])
                 : "v"(b[M & 7]), "v"(a[M >> 3]));
}

// Wait states before the accumulators of a run are read by vector instructions.
__device__ __forceinline__ void mfma_drain() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int MODE>
__device__ __forceinline__ void aim_at_tile(Copies<MODE>& c, const Tile& t, int w, int lane) {
  c.a.init(t.a, t.lda, t.a_rows, t.kl, w, lane);
  c.b.init(t.b, t.ldb, t.b_rows, t.kl, w, lane);
  c.stages = uni((t.kl + kStageK - 1) / kStageK);
}

// Begins a tile: the copies of its first two stages, into the two buffers.
template <int MODE>
__device__ __forceinline__ void begin_tile(Copies<MODE>& c, uint32_t lds, const Tile& t, int w,
                                           int lane) {
  aim_at_tile(c, t, w, lane);
  if (c.stages == 0) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    c.lds = uni(lds + s * kBufBytes + w * 1024);
    c.begin(s);
    static_for<kCopies>([&](auto q) {
      constexpr int P = decltype(q)::value;
      c.template copy_end<P>(c.template copy_begin<P>());
    });
  }
}

// A tile's contraction, begun by begin_tile.  stored: the epilogue of the tile before
// came after those copies, with at least kEpilogueStores stores (INT8: between them, 16 after
// the first stage's).
template <int MODE> constexpr int kEpilogueStores = MODE == kInt8 ? 16 : 32;

template <int MODE, bool F16>
__device__ __forceinline__ void contract(Copies<MODE>& c, uint32_t lds, int w, int lane,
                                         bool stored, v4f (&acc)[8][8]) {
  c.stages = uni(c.stages);
  if (c.stages == 0) return;
  c.a.make_uniform();
  c.b.make_uniform();
  using FragsA = FragOff<kColsA<MODE>, BM, 8>;
  using FragsB = FragOff<kColsB<MODE>, BN, 8>;
  FragsA fa;
  FragsB fb;
  fa.init(lds, (w >> 1) * 128, lane);
  fb.init(lds + kTileBytes, (w & 1) * 128, lane);
  c.lds = uni(lds + w * 1024);
  if (stored) wait_and_barrier<kCopies + kEpilogueStores<MODE>>();
  else wait_and_barrier<kCopies>();
  Half a0, b0, a1, b1;
  static_for<16>([&](auto q) { read_frag<MODE, 0, decltype(q)::value>(fa, fb, a0, b0); });
  int other = kBufBytes;  // bytes to the other buffer
  for (int kt = 0; kt < c.stages; ++kt) {
    c.begin(kt + 2);
    int voff = 0;
    fence();
    static_for<128>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      if constexpr (m < 64) mfma<MODE, F16, m>(a0, b0, acc);
      else mfma<MODE, F16, m - 64>(a1, b1, acc);
      fence();
      // the second half's fragments
      if constexpr (m < 32 && m % 2 == 0) read_frag<MODE, 1, m / 2>(fa, fb, a1, b1);
      // every wave has read this buffer
      if constexpr (m == kFreeSlot) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      // the reads move to the other buffer
      if constexpr (m > kFreeSlot && m % 2 == 1) {
        constexpr int q = (m - kFreeSlot) / 2;
        if constexpr (q < FragsA::kRegs) fa.template move<q>(other);
        else if constexpr (q < FragsA::kRegs + FragsB::kRegs)
          fb.template move<q - FragsA::kRegs>(other);
      }
      // the other buffer holds the next stage for every wave
      if constexpr (m == kReadySlot)
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kCopiesBeforeReady) : "memory");
      // the next stage's first half's fragments
      if constexpr (m >= kReadySlot && m < kReadySlot + 32 && m % 2 == 0)
        read_frag<MODE, 0, (m - kReadySlot) / 2>(fa, fb, a0, b0);
      // the stage after next into this buffer
      constexpr int cb = m + 1 - kCopySlot, ce = m - kCopySlot;
      if constexpr (ce >= 0 && ce % kCopyStep == 0 && ce / kCopyStep < kCopies)
        c.template copy_end<ce / kCopyStep>(voff);
      if constexpr (cb >= 0 && cb % kCopyStep == 0 && cb / kCopyStep < kCopies)
        voff = c.template copy_begin<cb / kCopyStep>();
      fence();
    });
    c.lds += other;
    other = -other;
  }
  fence();
  mfma_drain();
  fence();
}

// INT8: a tile's output, with the 32 copies of the next tile's first two stages (MORE) between
// its 32 pairs of blocks: copies and stores keep the memory path busy where the vector units
// alone would (a contraction is half as long as a 16-bit one's, and the end of a tile, copies and
// then stores, took 13 000 of its 87 000 cycles at k = 4096).  scales: of the tile's rows, then
// of its columns, in LDS.
// WHOLE: the tile has all its columns, so that a store's place is the row of blocks' and a constant.
// All of it is in the lane's offset: of the scalar one the compiler's description of these stores
// says that the range check, which drops the rows past the tile's, leaves it out.  (Rows in the
// scalar offset save an addition a row of blocks, and no time.)
template <bool F16, bool F32, bool WHOLE, bool MORE>
__device__ __forceinline__ void store_int8(const v4f (&acc)[8][8], const OutTile& o,
                                           const float* scales, int wrow, int wcol, int w,
                                           int lane, Copies<kInt8>& c, uint32_t lds) {
  constexpr int esz = F32 ? 4 : 2;
  static_assert(!(WHOLE && F32), "16-bit outputs");
  int ldo = o.ldo;
  asm volatile("" : "+s"(ldo));  // keeps all the store offsets from being hoisted
  const __amdgpu_buffer_rsrc_t ro = make_rsrc(o.out, (int64_t)o.rows * o.ldo * esz);
  const int q = lane >> 4, row = wrow + (lane & 15);
  int place = (row * ldo + wcol + 16 * (q & 1) + 8 * (q >> 1)) * 2;
  v4f cscale[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    cscale[j] = *reinterpret_cast<const v4f*>(scales + BM + wcol + 16 * j + 4 * q);
  static_for<8>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    const float rscale = scales[row + 16 * i];
    static_for<4>([&](auto jc) {
      constexpr int j = 2 * decltype(jc)::value, P = 4 * i + decltype(jc)::value;
      int voff = 0;
      fence();
      if constexpr (MORE) {
        if constexpr (P % kCopies == 0) {
          constexpr int S = P / kCopies;
          c.lds = uni(lds + S * kBufBytes + w * 1024);
          c.begin(S);
        }
        voff = c.template copy_begin<P % kCopies>();
      }
      fence();
      v4f y0 = acc[i][j], y1 = acc[i][j + 1];
      asm volatile("" : "+v"(y0), "+v"(y1));
      const v4i s0 = __builtin_bit_cast(v4i, y0), s1 = __builtin_bit_cast(v4i, y1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y0[e] = ((float)s0[e] * rscale) * cscale[j][e];
        y1[e] = ((float)s1[e] * rscale) * cscale[j + 1][e];
      }
      if constexpr (MORE) c.template copy_end<P % kCopies>(voff);
      if constexpr (WHOLE) {
        __builtin_amdgcn_raw_buffer_store_b128(swap_pair<F16>(y0, y1), ro, place + 32 * j, 0, 0);
      } else {
        store_pair<F32, F16>(y0, y1, ro, ldo, row + 16 * i, wcol + 16 * j, q, o.cols);
      }
      fence();
    });
    if constexpr (WHOLE) place += 32 * ldo;
  });
}

template <bool F16, bool MORE>
__device__ __forceinline__ void store_tile_int8(const v4f (&acc)[8][8], const OutTile& o,
                                                int out_f32, const float* scales, int wrow,
                                                int wcol, int w, int lane, Copies<kInt8>& c,
                                                uint32_t lds) {
  if (out_f32)
    store_int8<F16, true, false, MORE>(acc, o, scales, wrow, wcol, w, lane, c, lds);
  else if (o.cols == BN)
    store_int8<F16, false, true, MORE>(acc, o, scales, wrow, wcol, w, lane, c, lds);
  else
    store_int8<F16, false, false, MORE>(acc, o, scales, wrow, wcol, w, lane, c, lds);
}

// A tile's copies are begun before the epilogue of the one before it (INT8: in it), so that
// they arrive while that one's stores go out.
template <int MODE, bool F16>
__global__ __launch_bounds__(kThreads) void large_kernel(Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * kBufBytes];
  __shared__ Sched sm;
  __shared__ int ids[MODE == kLora ? BM : 1];
  __shared__ __attribute__((aligned(16))) float scales[MODE == kInt8 ? BM + BN : 4];
  const uint32_t lds = lds_offset(ring);
  const int total = count_tiles<MODE, BM, BN>(p, sm);
  const Rounds rounds = plan_rounds<MODE, false>(p, total);
  const int nsplit = rounds.nsplit;
  Work work = take_work(p, rounds, 0);
  if (work.tile < 0) return;
  Tile t = find_tile<MODE, BM, BN>(p, sm, uni(work.tile));
  if (work.part >= 0) narrow_tile<MODE>(t, uni(work.part), nsplit);
  Copies<MODE> c;
  begin_tile(c, lds, t, uni((int)(threadIdx.x >> 6)), threadIdx.x & 63);
  bool stored = false;
  for (int round = 1;; ++round) {
    // opaque per-tile copy of the thread index: keeps the offsets of the tile body
    // from being hoisted out of the persistent loop
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, w = uni(tid >> 6);
    const int wrow = (w >> 1) * 128, wcol = (w & 1) * 128;
    v4f acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        asm volatile("" : "+a"(acc[i][j]));
      }
    if constexpr (MODE == kLora) tile_adapters<BM>(p, sm, t, ids);
    float rscale = 0.0f, cscale = 0.0f;
    if constexpr (MODE == kInt8) {
      // a row and a column a thread; they arrive during the contraction
      if (tid < t.a_rows) rscale = p.a_scales[t.row0 + tid];
      if (tid < t.b_rows) cscale = p.b_scales[t.col0 + tid];
    }
    contract<MODE, F16>(c, lds, w, lane, stored, acc);
    if constexpr (MODE == kInt8) {
      scales[tid] = rscale;
      scales[BM + tid] = cscale;
    }
    // every copy has landed and no wave still reads a buffer before the next
    // tile's first copies
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const Work next = take_work(p, rounds, round);
    Tile tn = t;
    if (next.tile >= 0) {
      tn = find_tile<MODE, BM, BN>(p, sm, uni(next.tile));
      if (next.part >= 0) narrow_tile<MODE>(tn, uni(next.part), nsplit);
      if (MODE == kInt8 && work.part < 0) aim_at_tile(c, tn, w, lane);
      else begin_tile(c, lds, tn, w, lane);
    }
    if constexpr (MODE == kLora) {
      add_low_rank<F16, 8, 8>(p, t, ids, wrow, wcol, lane, uni(work.part), work.nparts, acc);
      __syncthreads();  // ids are read before the next tile's
    }
    if (work.part >= 0) {
      write_split_record<MODE>(p.ws, work.slot, nsplit, t);
      store_part<8, 8>(
          reinterpret_cast<float*>(p.ws + kWsHeader + (int64_t)work.slot * kPartBytes), acc, w,
          lane, wrow, t.a_rows);
    } else if constexpr (MODE == kInt8) {
      const OutTile o = out_tile<MODE>(p, t);
      if (next.tile >= 0)
        store_tile_int8<F16, true>(acc, o, p.out_f32, scales, wrow, wcol, w, lane, c, lds);
      else
        store_tile_int8<F16, false>(acc, o, p.out_f32, scales, wrow, wcol, w, lane, c, lds);
    } else {
      store_blocks<MODE, F16, 8, 8>(acc, out_tile<MODE>(p, t), p.out_f32, wrow, wcol, lane);
    }
    if (next.tile < 0) break;
    stored = work.part < 0;
    work = next;
    t = tn;
  }
}

template <int MODE, bool F16>
hipError_t launch(Args p, hipStream_t stream) {
  const int grid = prepare_launch<MODE, BM, BN>(p, device_cu_count());
  if (grid == 0) return hipSuccess;
  hipLaunchKernelGGL((large_kernel<MODE, F16>), dim3(grid), dim3(kThreads), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.ws == nullptr) return e;
  hipLaunchKernelGGL((split_reduce_kernel<MODE == kInt8, F16, BM, BN, 2, 8, 8>),
                     dim3(reduce_grid(grid, BM * BN / 512)), dim3(kThreads), 0, stream, p.ws, p.out,
                     p.c, p.ldo, p.out_f32, p.a_scales, p.b_scales);
  return hipGetLastError();
}

}  // namespace large
}  // namespace g16
}  // namespace bsg

#endif  // BSG_GEMM_LARGE_H
