// Parts shared by the kernels of the 16-bit grouped products (bf16 or fp16
// operands, FP32 accumulation):
//
//   FPROP_TN:  Y[r, :]  = C[r, :] + A[r, :] B_g^T      r in group g
//   DGRAD_NN:  Y[r, :]  = C[r, :] + A[r, :] B_g        r in group g
//   WGRAD_NT:  Y_g      = C_g + A_g^T B_g              over the group's rows
//
// and, beside a projection shared by all rows, the low-rank product of each
// row's own adapter (LORA): Y[r, :] = A[r, :] B^T + low[r, :] U_a^T.
//
// Every output tile is one contraction of an A tile and a B tile.  An operand
// lies in memory either with the contraction innermost ("rows": both operands
// of FPROP, A of DGRAD) or with its rows innermost ("columns": B of DGRAD, both
// of WGRAD).  Both kinds are copied to LDS as they lie, 64 contraction indexes a
// stage, in whole lines; the transposition that the matrix instruction needs of
// the second kind is done by the LDS reads (ds_read_b64_tr_b16), so no operand
// is transposed in memory and none passes through the vector units.
//
// LDS layout of an operand tile of BR rows (both kinds take 128 BR bytes):
//   rows:    row r at 128 r; 16-byte chunk c (8 contraction indexes) in slot
//            c ^ ((r / 2) % 8), so that 16 lanes reading one chunk of 16
//            consecutive rows hit all 64 banks.
//   columns: contraction index k at 2 BR k; chunk c (8 rows) in slot
//            c ^ swz(k), so that the eight 32-byte pieces that 32 lanes of a
//            transposing read take (k = 0 .. 3 and 8 .. 11 of a step) hit all 64
//            banks.
//
// Matrix instruction: v_mfma_f32_16x16x32, lane (r, q) = (l % 16, l / 16) holds
// contraction indexes 8 q .. 8 q + 7 of row r.  B is its first operand and A its
// second, so lane (r, q) ends with output row r, columns 4 q + [0, 4) of a
// 16 x 16 block.  On this chip products of random operands are limited by power:
// a loop of these instructions alone runs at 2.06 PFLOP/s (2.04 GHz), one of
// v_mfma_f32_32x32x16 at 1.78 (1.73 GHz), and both at 2.45 on zeros.
#ifndef BSG_GEMM_16BIT_H
#define BSG_GEMM_16BIT_H

#include <utility>

#include "bsg_internal.h"
#include "lds_dma.h"
#include "store_tile.h"

namespace bsg {
namespace g16 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kStageK = 64;       // contraction indexes per LDS stage
constexpr int kThreads = 256;
constexpr int kSuperM = 4, kSuperN = 8;  // tile block one XCD works on
constexpr int kLowParts = 4;             // of the adapters' first product, where it is split
constexpr int kLowValues = 3;            // 16-bit values that carry a sum of it to the second
constexpr int kLowChunk = 64;            // rank columns that share a row's power of two

enum Mode { kFprop = 0, kWgrad = 1, kDgrad = 2, kLora = 3, kInt8 = 4 };
template <int MODE> constexpr bool kColsA = MODE == kWgrad;
template <int MODE> constexpr bool kColsB = MODE == kWgrad || MODE == kDgrad;

template <typename F, int... Is>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Division of a < 2^31 by a number that the host knows: m = ceil(2^(31 + s) / d) with
// 2^s >= d > 2^(s - 1) gives a / d as the high half of m * 2 a, shifted by s.  What
// stands before a tile's first copy is short calls' latency, and an inlined division is
// some 30 instructions to fetch.
struct Div {
  uint32_t m, s, d;
};
inline Div make_div(int64_t d) {
  Div v{0, 0, (uint32_t)d};
  while (((int64_t)1 << v.s) < d) ++v.s;
  v.m = (uint32_t)((((uint64_t)1 << (31 + v.s)) + (uint64_t)d - 1) / (uint64_t)d);
  return v;
}
__device__ __forceinline__ int div_by(int a, const Div& v) {
  return (int)(__umulhi(v.m, 2u * (uint32_t)a) >> v.s);
}
// a / b of small numbers (a < 2^20, b >= 1): the float quotient is off by less than one
// step of 1 / b at a whole number.
__device__ __forceinline__ int div_small(int a, int b) {
  return (int)(((float)a + 0.5f) * __builtin_amdgcn_rcpf((float)b));
}

struct Args {
  const uint16_t* a;
  const uint16_t* b;
  const int64_t* offsets;
  const char* c;
  char* out;
  int64_t lda, ldb, stride_b, ldo, stride_o;  // elements
  int64_t rows_cap, n, k;
  uint32_t* status;
  char* ws;  // split workspace or null: no split
  int G, out_f32;
  Div grid, band;  // workgroups; tiles of kSuperM rows of tiles
  // LORA
  void* low;               // X A^T of each row's own adapter: 16-bit [rows_cap, kLowValues, r],
                           // the values that carry it, or (low_parts: kLowParts, not 1)
                           // float32 [kLowParts, rows_cap, r], parts of its contraction
  float* low_power;        // fp16, low_parts 1: [rows_cap, r / kLowChunk rounded up], the power
                           // of two to multiply the values of a row's chunk by
  const float* scale;      // [adapters]
  int low_parts;
  const uint16_t* up;      // [adapters, n, r]
  const int32_t* adapter;  // [G], negative: none
  int num_adapters, r;
  // INT8
  const float* a_scales;   // [rows_cap]
  const float* b_scales;   // [G, n]
};

struct Sched {
  int64_t off[kMaxGroups + 1];
  int32_t cnt[kMaxGroups];  // tiles of each group; LORA: adapter of each request, or -1
  int32_t pre[kMaxGroups + 1];
};

struct Tile {
  const uint16_t* a;  // first element of the operand tiles
  const uint16_t* b;
  int64_t lda, ldb;
  int a_rows, b_rows;  // live rows (those past them read as zeros)
  int kl;              // contraction length
  int64_t out_off;     // bytes from out (and c) to the tile's first element
  int64_t row0;        // LORA, INT8: first row
  int64_t col0;        // LORA: first column; INT8: of all groups' columns
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uni64(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v & 0xffffffff));
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

template <typename T>
__device__ __forceinline__ uint32_t lds_offset(T* shared_ptr) {
  return (uint32_t)(size_t)(__attribute__((address_space(3))) T*)(shared_ptr);
}

__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Vector-memory operations complete in issue order: waits until only the N most
// recent are outstanding and for this wave's LDS accesses, then joins the barrier.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- tiles

// Adapter of request g, or -1.
__device__ __forceinline__ int adapter_of(const Args& p, int g) {
  const int a = p.adapter[g];
  return a < p.num_adapters ? a : -1;
}

// Loads the offsets and counts tiles; returns their number.  Every thread calls it.
template <int MODE, int BM, int BN>
__device__ __forceinline__ int count_tiles(const Args& p, Sched& sm) {
  const int tid = threadIdx.x;
  if constexpr (MODE == kLora) {
    for (int g = tid; g < p.G; g += kThreads) sm.cnt[g] = adapter_of(p, g);
  }
  load_offsets_clamped(p.offsets, p.G, p.rows_cap, sm.off, blockIdx.x == 0 ? p.status : nullptr);
  const int64_t ntn = (p.n + BN - 1) / BN;
  if constexpr (MODE == kLora) {
    // all rows of all requests are one run of rows of the shared projection
    __syncthreads();
    const int64_t m = sm.off[p.G] - sm.off[0];
    const int total = (int)(((m > 0 ? m : 0) + BM - 1) / BM * ntn);
    return uni(total);
  } else {
    for (int g = tid; g < p.G; g += kThreads)
      sm.cnt[g] = (int32_t)(MODE == kWgrad ? ((p.n + BM - 1) / BM) * ((p.k + BN - 1) / BN)
                                           : ((group_extent(sm.off, g) + BM - 1) / BM) * ntn);
    __syncthreads();
    wave0_exclusive_scan(sm.cnt, p.G, sm.pre);
    __syncthreads();
    return uni(sm.pre[p.G]);
  }
}

// Position (mt, nt) of tile u of mtiles x ntiles, as super_tile has it; band divides by
// kSuperM * ntiles.
__device__ __forceinline__ void place_tile(int u, int mtiles, int ntiles, const Div& band, int& mt,
                                           int& nt) {
  static_assert(kSuperM == 4 && kSuperN == 8, "shifts");
  const int full_rows = mtiles >> 2;
  int br = full_rows, hgt = mtiles & 3;
  if (u < full_rows * (4 * ntiles)) {
    br = div_by(u, band);
    hgt = 4;
  }
  u -= br * (4 * ntiles);
  const auto by_hgt = [hgt](uint32_t v) {  // 1, 2, 3 or 4
    return hgt == 3 ? __umulhi(v, 0x55555556u) : v >> (hgt >> 1);
  };
  const int bc = (int)by_hgt((uint32_t)u >> 3);
  u -= bc * (8 * hgt);
  const int q = (int)by_hgt((uint32_t)u);
  mt = br * 4 + u - q * hgt;
  nt = bc * 8 + q;
}

template <int MODE, int BM, int BN>
__device__ __forceinline__ Tile find_tile(const Args& p, const Sched& sm, int tile) {
  const int esz = p.out_f32 ? 4 : 2;
  Tile t;
  int mt, nt;
  if constexpr (MODE == kWgrad) {
    const int g = uni(find_group(sm.pre, p.G, tile));
    place_tile(tile - uni(sm.pre[g]), (int)((p.n + BM - 1) / BM), (int)((p.k + BN - 1) / BN),
               p.band, mt, nt);
    const int64_t i0 = (int64_t)mt * BM, j0 = (int64_t)nt * BN;
    const int64_t t0 = uni64(sm.off[g]);
    t.a = p.a + t0 * p.lda + i0;
    t.b = p.b + t0 * p.ldb + j0;
    const int64_t rv = p.n - i0, cv = p.k - j0;
    t.a_rows = (int)(rv < BM ? rv : BM);
    t.b_rows = (int)(cv < BN ? cv : BN);
    t.kl = uni((int)group_extent(sm.off, g));
    t.out_off = (g * p.stride_o + i0 * p.ldo + j0) * esz;
    t.row0 = t.col0 = 0;
  } else {
    const int g = MODE == kLora ? 0 : uni(find_group(sm.pre, p.G, tile));
    const int64_t first = uni64(sm.off[g]);
    const int64_t m = MODE == kLora ? uni64(sm.off[p.G]) - first : uni64(group_extent(sm.off, g));
    place_tile(MODE == kLora ? tile : tile - uni(sm.pre[g]), (int)((m + BM - 1) / BM),
               (int)((p.n + BN - 1) / BN), p.band, mt, nt);
    const int64_t r0 = (int64_t)mt * BM, n0 = (int64_t)nt * BN;
    t.a = p.a + (first + r0) * p.lda;
    t.b = p.b + (MODE == kLora ? 0 : g * p.stride_b) + (MODE == kDgrad ? n0 : n0 * p.ldb);
    const int64_t rv = m - r0, cv = p.n - n0;
    t.a_rows = (int)(rv < BM ? rv : BM);
    t.b_rows = (int)(cv < BN ? cv : BN);
    t.kl = (int)p.k;
    t.out_off = ((first + r0) * p.ldo + n0) * esz;
    t.row0 = first + r0;
    t.col0 = MODE == kInt8 ? g * p.n + n0 : n0;
  }
  t.lda = p.lda;
  t.ldb = p.ldb;
  return t;
}

// ---------------------------------------------------------------- global -> LDS

template <int BR>
__device__ __forceinline__ int swz(int k) {
  static_assert(BR >= 128, "a row of 16 chunks or more");
  return 4 * (k & 3) + 2 * ((k >> 3) & 1);
}

// A global -> LDS copy of 16 bytes a lane (1 KiB at `at` + IMM) in two steps, so that
// other instructions can stand between them: the load has to be a wait state later
// than the writing of m0, which nothing else reads.  MASKED: the lane's offset is
// past every range for lanes outside of `mask`.
template <int IMM, bool MASKED>
__device__ __forceinline__ int copy16_begin(uint32_t at, int voff, uint64_t mask) {
  if constexpr (MASKED) {
    int o;
    asm volatile(
        "s_add_u32 m0, %1, %2\n\t"
        "v_cndmask_b32 %0, %3, %4, %5"
        : "=v"(o)
        : "s"(at), "n"(IMM), "v"(kDmaOutOfRange), "v"(voff), "s"(mask)
        : "memory", "scc");
    return o;
  } else {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0" : : "s"(at), "n"(IMM) : "memory", "scc");
    return voff;
  }
}
__device__ __forceinline__ void copy16_end(const v4i& rsrc, int voff) {
  asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(rsrc) : "memory");
}

// One wave's share of the copies of an operand tile of BR rows: pieces w, w + 4,
// .. of the tile's BR / 8 pieces of 1 KiB.
//   rows:    piece p is rows 8 p .. 8 p + 7, lane l row 8 p + l / 8, slot l % 8
//   columns: piece p is 512 / BR contraction indexes, lane l index l / (BR / 8)
//            of them, slot l % (BR / 8)
// A stage's descriptor begins at the stage, so a lane's offsets are the same in
// every stage.  What lies past the tile's rows or the contraction is copied as
// zeros: by the descriptor's range, by a column's offset past every range, or (rows,
// a last stage that is not whole) by the stage's lane mask.
template <bool COLS, int BR>
struct Side {
  static constexpr int kPieces = BR / 32;  // per wave
  uint64_t base;
  int range;  // rows: bytes of the whole tile
  int ld2;    // bytes between memory rows
  int kl;
  uint64_t last;  // rows: lanes whose chunk lies within the contraction in the last stage
  int off[kPieces];

  __device__ __forceinline__ void init(const uint16_t* src, int64_t ld, int rows, int contraction,
                                       int w, int lane) {
    base = (uint64_t)uni64((int64_t)reinterpret_cast<uint64_t>(src));
    ld2 = uni((int)(ld * 2));
    kl = uni(contraction);
    if constexpr (!COLS) {
      const int row = 8 * w + (lane >> 3);
      const int c = (lane & 7) ^ ((row >> 1) & 7);
      range = uni(rows) * ld2;
      last = __ballot(c * 8 < kl - (kl - 1) / kStageK * kStageK);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) off[i] = (row + 32 * i) * ld2 + c * 16;
    } else {
      constexpr int cpr = BR / 8, rpp = 512 / BR;
      range = 0;
      last = 0;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int k = rpp * (w + 4 * i) + lane / cpr;
        const int c = (lane % cpr) ^ swz<BR>(k);
        off[i] = c * 8 < rows ? k * ld2 + c * 16 : kDmaOutOfRange;
      }
    }
    // a buffer instruction has to be five wait states later than the vector
    // instructions that wrote its descriptor, which the compiler does not know of
    // instructions in asm
    asm volatile("s_nop 4" : "+s"(base), "+s"(range), "+s"(ld2));
  }

  // Says again that what is uniform is (it is carried from one tile to the next).
  __device__ __forceinline__ void make_uniform() {
    base = (uint64_t)uni64((int64_t)base);
    range = uni(range);
    ld2 = uni(ld2);
    kl = uni(kl);
    last = (uint64_t)uni64((int64_t)last);
  }

  // Lanes whose chunk lies within the contraction in stage kt of `stages`.
  __device__ __forceinline__ uint64_t mask(int kt, int stages) const {
    return kt == stages - 1 ? last : ~0ull;
  }

  // Descriptor of stage kt (nothing is in range when it is not live).
  __device__ __forceinline__ v4i rsrc(int kt, bool live) const {
    const int64_t at = (int64_t)kt * (COLS ? kStageK * (int64_t)ld2 : 2 * kStageK);
    const int left = kl - kt * kStageK;
    const int bytes =
        !live ? 0 : COLS ? (left < kStageK ? left : kStageK) * ld2 : range - kt * 2 * kStageK;
    const uint64_t p = base + (uint64_t)at;
    return v4i{(int)(uint32_t)p, (int)(uint32_t)(p >> 32), bytes, 0x00020000};
  }

  template <int I, int IMM>
  __device__ __forceinline__ int copy_begin(uint32_t at, uint64_t m) const {
    return copy16_begin<IMM, !COLS>(at, off[I], m);
  }
  template <int I, int IMM>
  __device__ __forceinline__ void copy(const v4i& rs, uint32_t at, uint64_t m) const {
    copy16_end(rs, copy_begin<I, IMM>(at, m));
  }
};

// ---------------------------------------------------------------- LDS -> registers

// Offsets of a lane's fragment reads: one register a half stage of 32 indexes
// (rows; the 16-row steps are immediates) or a 16-row block (columns; the half
// stages are).
template <bool COLS, int BR, int NB>
struct FragOff {
  static constexpr int kRegs = COLS ? NB : 2;
  int o[kRegs];
  // tile: the operand's LDS; row0: the wave's first row
  __device__ __forceinline__ void init(uint32_t tile, int row0, int lane) {
    const int r = lane & 15, q = lane >> 4;
    if constexpr (!COLS) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        o[s] = (int)tile + (row0 + r) * 128 + (((4 * s + q) ^ ((r >> 1) & 7)) << 4);
    } else {
      const int k = 8 * q + (r >> 2);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int c = (row0 >> 3) + 2 * i + ((lane & 3) >> 1);
        o[i] = (int)tile + k * (BR * 2) + ((c ^ swz<BR>(k)) << 4) + 8 * (lane & 1);
      }
    }
#pragma unroll
    for (int t = 0; t < kRegs; ++t) asm volatile("" : "+v"(o[t]));
  }
  template <int T>
  __device__ __forceinline__ void move(int bytes) {
    o[T] += bytes;
  }
  // Rows 16 I + lane % 16, contraction indexes 32 S + 8 (lane / 16) + [0, 8).
  // at: bytes from the tile given to init.
  template <int I, int S>
  __device__ __forceinline__ v4i read(uint32_t at = 0) const {
    if constexpr (!COLS) {
      return *reinterpret_cast<const lds_v4i*>((size_t)(uint32_t)(o[S] + at + I * 2048));
    } else {
      const uint32_t p = o[I] + at + S * 64 * BR;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(size_t)p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(size_t)(p + 8 * BR));
      const v2i l = __builtin_bit_cast(v2i, lo), u = __builtin_bit_cast(v2i, hi);
      return v4i{l[0], l[1], u[0], u[1]};
    }
  }
};

template <bool F16>
__device__ __forceinline__ v4f mfma16(const v4i& x, const v4i& y, const v4f& acc) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x),
                                                  __builtin_bit_cast(v8h, y), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x),
                                                   __builtin_bit_cast(v8bf, y), acc, 0, 0, 0);
}

template <int MODE, bool F16>
__device__ __forceinline__ v4f mfma_step(const v4i& x, const v4i& y, const v4f& acc) {
  if constexpr (MODE == kInt8)
    return __builtin_bit_cast(
        v4f, __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, __builtin_bit_cast(v4i, acc), 0, 0, 0));
  else
    return mfma16<F16>(x, y, acc);
}

// ---------------------------------------------------------------- adapters

// Request of a row in [off[0], off[G]).
__device__ __forceinline__ int request_of(const int64_t* off, int G, int64_t row) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <bool F16>
__device__ __forceinline__ float to_f32(uint32_t b) {
  return F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)b) : bf16_to_f32(b & 0xffffu);
}

// The sums x A^T go into the second product as 16-bit values whose sum they are.  A bf16
// value has float32's range, so the values are the nearest one to the sum, the nearest to
// what is left of it and what is left then.  An fp16 value has 40 binades with its
// subnormals, so
//   - the rank columns of a row's chunk are divided by a power of two that puts the largest
//     into [2^14, 2^15), and the products multiplied by it again, and
//   - what the first value leaves is held times 2^11 and its products are summed apart, so
//     that it reaches below fp16's smallest values.
// Both are exact.  So the second product takes the sum as float32 has it, all 24 bits: three
// values of 8 or 11 bits are what that takes.  (fp16: of a sum that is under 2^-26 of the
// largest in its row's chunk, what lies above 2^-50 of that.)
//
// low_scales: multiplies by `down` before and `up` after, for a chunk's largest magnitude m
// (zero, infinite and NaN too).
struct LowScales {
  float down, up;
};
__device__ __forceinline__ LowScales low_scales(float m) {
  int e = (int)(__float_as_uint(m) >> 23 & 255u);
  if (e < 15) e = 15;  // both powers stay normal numbers
  return {__uint_as_float((uint32_t)(268 - e) << 23), __uint_as_float((uint32_t)(e - 14) << 23)};
}

constexpr float kRestScale = 2048.0f;  // fp16: of the values after the first

// Two sums, in place of the low and the high half of each word.  A value that others follow
// is kept finite, so that an infinity stays one in the last and does not turn into the
// difference of two (a NaN passes the same way: the median of a NaN is a number).
template <bool F16>
__device__ __forceinline__ void split_low(float a, float b, uint32_t (&word)[kLowValues]) {
  constexpr float kMax = F16 ? 65504.0f : 3.3895313892515355e38f;
#pragma unroll
  for (int h = 0; h < kLowValues - 1; ++h) {
    word[h] = pack16<F16>(__builtin_amdgcn_fmed3f(a, -kMax, kMax),
                          __builtin_amdgcn_fmed3f(b, -kMax, kMax));
    a -= to_f32<F16>(word[h] & 0xffffu);
    b -= to_f32<F16>(word[h] >> 16);
    if (F16 && h == 0) {
      a *= kRestScale;
      b *= kRestScale;
    }
  }
  word[kLowValues - 1] = pack16<F16>(a, b);
}

// A lane's fragments of a 16-row block's low values: `row` of the wave's rows, 32 rank columns
// and 32 more, each from byte 2 * column = at[c] on (an offset past every range: zeros), all
// of the chunk that begins at column k.  Returns what the products have to be multiplied by.
// rows: live rows from the wave's first on; halves: 1 leaves the second fragments alone.
template <bool F16>
__device__ __forceinline__ float load_low(const Args& p, int64_t first, int rows, int row, int k,
                                          int halves, const uint32_t (&at)[2],
                                          v4i (&v)[2][kLowValues]) {
  const int rank = p.r;
  if (p.low_parts == 1) {
    const int line = 2 * kLowValues * rank;
    const __amdgpu_buffer_rsrc_t low =
        make_rsrc(static_cast<uint16_t*>(p.low) + first * kLowValues * rank,
                  rows > 0 ? rows * line : 0);
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int h = 0; h < kLowValues; ++h)
        v[c][h] = __builtin_amdgcn_raw_buffer_load_b128(
            low, (int)(at[c] + row * line + 2 * h * rank), 0, 0);
    if constexpr (!F16) return 1.0f;
    const int chunks = (rank + kLowChunk - 1) / kLowChunk;
    const __amdgpu_buffer_rsrc_t power =
        make_rsrc(p.low_power + first * chunks, rows > 0 ? rows * chunks * 4 : 0);
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        power, 4 * (row * chunks + k / kLowChunk), 0, 0));
  }
  float s[2][8];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[c][e] = 0.0f;
    if (c >= halves) continue;
    const uint32_t o = at[c] == (uint32_t)kDmaOutOfRange ? at[c] : 2 * at[c] + row * 4 * rank;
    v4i part[kLowParts][2];
#pragma unroll
    for (int i = 0; i < kLowParts; ++i) {
      const __amdgpu_buffer_rsrc_t low =
          make_rsrc(static_cast<float*>(p.low) + (i * p.rows_cap + first) * rank,
                    rows > 0 ? rows * 4 * rank : 0);
#pragma unroll
      for (int b = 0; b < 2; ++b)
        part[i][b] = __builtin_amdgcn_raw_buffer_load_b128(low, (int)(o + 16 * b), 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[c][e] = __int_as_float(part[0][e >> 2][e & 3]);
#pragma unroll
      for (int i = 1; i < kLowParts; ++i) s[c][e] += __int_as_float(part[i][e >> 2][e & 3]);
    }
  }
  LowScales f{1.0f, 1.0f};
  if constexpr (F16) {
    // the row's other columns are in the lanes 16, 32 and 48 further
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(s[e >> 3][e & 7]));
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    f = low_scales(m);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (c >= halves) continue;  // what v holds there is not used
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t word[kLowValues];
      split_low<F16>(s[c][2 * e] * f.down, s[c][2 * e + 1] * f.down, word);
#pragma unroll
      for (int h = 0; h < kLowValues; ++h) v[c][h][e] = (int)word[h];
    }
  }
  return f.up;
}

constexpr int kWaitLoads = 0x0f70;  // s_waitcnt vmcnt(0)

// Adds each row's own low-rank product to a wave's accumulators: for every
// adapter that occurs in (64 of) the wave's rows one product of the rows' low values
// with the adapter's rows of `up`, kept for its own rows only.  So what
// an adapter holds (infinities, NaN) never reaches a row of another request, and the
// cost follows the adapters that meet in the wave's rows, not the requests.  The
// operands come straight from the L2, 64 rank columns at a time, the low values
// once and `up` once an adapter, so that a load's latency is paid per adapter and
// not per block.
// ids: adapter of each of the tile's rows (-1: none).  A split tile's parts share
// the adapters out: the c-th of the rows goes to part c % nparts.
template <bool F16, int MI, int NJ>
__device__ __forceinline__ void add_low_rank(const Args& p, const Tile& t, const int* ids, int wrow,
                                             int wcol, int lane, int part, int nparts,
                                             v4f (&acc)[MI][NJ]) {
  constexpr int kI = MI < 4 ? MI : 4, kJ = NJ < 4 ? NJ : 4;
  const int q = lane >> 4, rank = p.r;
  // rows and columns past the tile's, and rank columns past the last, read as zeros
  const int cols = t.b_rows - wcol;
  for (int k = 0; k < rank; k += kLowChunk) {
    // opaque: keeps the offsets of all loads from being hoisted out of the loop
    int r = lane & 15;
    asm volatile("" : "+v"(r));
    // halves of the chunk that hold rank columns (one workgroup a compute unit has no scalar
    // registers to spare for the branches, and loses 1 % with them)
    const int halves = MI == 8 || rank - k > kLowChunk / 2 ? 2 : 1;
    uint32_t at[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = k + 32 * c + 8 * q;
      at[c] = col < rank ? 2 * col : kDmaOutOfRange;
    }
    static_for<MI / kI>([&](auto gc) {
      constexpr int i0 = decltype(gc)::value * kI;
      const int row0 = wrow + 16 * i0;
      const int id = lane < 16 * kI ? ids[row0 + lane] : -1;  // of row lane
      uint64_t todo = __ballot(id >= 0);
      // the next `count` adapters are others' to add
      const auto pass = [&](int count) {
        for (; count > 0 && todo != 0; --count)
          todo &= ~__ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(todo)));
      };
      pass(part);
      if (todo == 0) return;
      v4i l[kI][2][kLowValues];  // [block][32 rank columns]
      float factor[kI];          // of a row's products
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const int mine = ids[row0 + 16 * i + r];
        factor[i] =
            load_low<F16>(p, t.row0 + row0, t.a_rows - row0, 16 * i + r, k, halves, at, l[i]) *
            (mine >= 0 ? p.scale[mine] : 0.0f);
      }
      while (todo != 0) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t own = __ballot(id == a);
        todo &= ~own;
        pass(nparts - 1);
        const __amdgpu_buffer_rsrc_t up = make_rsrc(
            p.up + ((int64_t)a * p.n + t.col0 + wcol) * rank, cols > 0 ? cols * 2 * rank : 0);
        static_for<NJ / kJ>([&](auto hc) {
          constexpr int jh = decltype(hc)::value * kJ;
          fence();
          v4i u[2][kJ];
#pragma unroll
          for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              u[c][j] = __builtin_amdgcn_raw_buffer_load_b128(
                  up, (int)(at[c] + (16 * (jh + j) + r) * 2 * rank), 0, 0);
          static_for<kI>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            const uint32_t these = (uint32_t)(own >> (16 * i)) & 0xffffu;
            if (these == 0) return;
            const bool mine = (these >> r & 1) != 0;
            static_for<kJ / 2>([&](auto jc) {
              constexpr int j0 = decltype(jc)::value * 2, ja = jh + j0;
              fence();
              // fp16: the values after the first are summed apart
              constexpr int kSums = F16 ? 2 : 1;
              v4f one[kSums][2];
#pragma unroll
              for (int z = 0; z < 2 * kSums; ++z) one[z >> 1][z & 1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (c >= halves) continue;
#pragma unroll
                for (int h = kLowValues - 1; h >= 0; --h)
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    v4f& sum = one[h > 0 ? kSums - 1 : 0][j];
                    sum = mfma16<F16>(u[c][j0 + j], l[i][c][h], sum);
                  }
              }
              // opaque copies: the accumulators stay where they are between the adapters
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                v4f y = acc[i0 + i][ja + j];
                asm volatile("" : "+v"(y));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float all = F16 ? fmaf(one[kSums - 1][j][e], 1.0f / kRestScale, one[0][j][e])
                                        : one[0][j][e];
                  y[e] = mine ? fmaf(all, factor[i], y[e]) : y[e];
                }
                acc[i0 + i][ja + j] = y;
                if constexpr (MI * NJ == 64) asm volatile("" : "+a"(acc[i0 + i][ja + j]));
              }
              fence();
            });
          });
        });
      }
      // Waits for loads that no block has used.  Left outstanding, the compiler waits for
      // them where their registers are written again: in the contraction's loop, where that
      // waits for the copies in flight as well.
      __builtin_amdgcn_s_waitcnt(kWaitLoads);
    });
  }
}

// Fills ids[0..BM) for a tile; the caller places a barrier after it.
template <int BM>
__device__ __forceinline__ void tile_adapters(const Args& p, const Sched& sm, const Tile& t,
                                              int* ids) {
  for (int i = threadIdx.x; i < BM; i += kThreads)
    ids[i] = i < t.a_rows ? sm.cnt[request_of(sm.off, p.G, t.row0 + i)] : -1;
}

// ---------------------------------------------------------------- epilogue

// Where a tile's output goes: its first element, live rows and columns.
struct OutTile {
  char* out;
  const char* c;  // or null
  int ldo, rows, cols;
  const float* a_scales;  // INT8: of the tile's rows
  const float* b_scales;  // INT8: of its columns
};

// This lane's byte offset of a block's columns 4 q + [0, 4) in an output tile: a
// column past out_cols gets an offset past every range.
template <int ESZ>
__device__ __forceinline__ int block_off(int ldo, int row, int col, int out_cols) {
  return col < out_cols ? (row * ldo + col) * ESZ : (int)kDropped;
}

// The addend of one 16 x 16 block as it lies in memory, and as numbers.
template <bool F32>
struct Addend {
  v4i v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rc, int off) {
    if constexpr (F32) {
      v = __builtin_amdgcn_raw_buffer_load_b128(rc, off, 0, 0);
    } else {
      const v2i t = __builtin_amdgcn_raw_buffer_load_b64(rc, off, 0, 0);
      v[0] = t[0];
      v[1] = t[1];
    }
  }
  template <bool F16>
  __device__ __forceinline__ float at(int e) const {
    if constexpr (F32) return __int_as_float(v[e]);
    const uint32_t bits = ((uint32_t)v[e >> 1] >> (16 * (e & 1))) & 0xffffu;
    return F16 ? (float)__builtin_bit_cast(_Float16, (unsigned short)bits) : bf16_to_f32(bits);
  }
};

// Two neighbouring 16 x 16 blocks of accumulators, the first at column col0: this
// lane's row `row`, columns col0 + 16 b + 4 q + [0, 4).  Rows past the live ones
// are dropped by the descriptors' range.
//   float32: a store is 16 bytes a lane, 64-byte runs of 16 rows.
//   16-bit:  lanes trade halves of the two blocks (v_permlane16_swap), after which
//            lane (r, q) holds columns 8 (q / 2) + [0, 8) of block q % 2: 16 bytes
//            a lane, and again 64-byte runs of 16 rows.
template <bool F16>
__device__ __forceinline__ v4i swap_pair(const v4f& y0, const v4f& y1) {
  const auto lo = __builtin_amdgcn_permlane16_swap((int)pack16<F16>(y0[0], y0[1]),
                                                   (int)pack16<F16>(y1[0], y1[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((int)pack16<F16>(y0[2], y0[3]),
                                                   (int)pack16<F16>(y1[2], y1[3]), false, false);
  return v4i{(int)lo[0], (int)hi[0], (int)lo[1], (int)hi[1]};
}

template <bool F32, bool F16>
__device__ __forceinline__ void store_pair(const v4f& y0, const v4f& y1, __amdgpu_buffer_rsrc_t ro,
                                           int ldo, int row, int col0, int q, int out_cols) {
  if constexpr (F32) {
    const int col = col0 + 4 * q;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, y0), ro,
                                           block_off<4>(ldo, row, col, out_cols), 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, y1), ro,
                                           block_off<4>(ldo, row, col + 16, out_cols), 0, 0);
  } else {
    const int col = col0 + 16 * (q & 1) + 8 * (q >> 1);
    __builtin_amdgcn_raw_buffer_store_b128(swap_pair<F16>(y0, y1), ro,
                                           block_off<2>(ldo, row, col, out_cols), 0, 0);
  }
}

// A wave's MI x NJ blocks, the first at (wrow, wcol) of the tile, two at a time: the
// accumulators are copied out right before their stores.  The addend, if there is
// one, is added in float32 before the one rounding, and read a row of blocks ahead.
// INT8: a sum becomes a float32 number (one rounding), is multiplied by its row's scale,
// then by its column's.
template <int MODE, bool F16, bool F32, bool ADD, int MI, int NJ>
__device__ __forceinline__ void store_rows(const v4f (&acc)[MI][NJ], const OutTile& o, int wrow,
                                           int wcol, int lane) {
  static_assert(NJ % 2 == 0, "blocks are stored in pairs");
  constexpr int esz = F32 ? 4 : 2;
  int ldo = o.ldo;
  asm volatile("" : "+s"(ldo));  // keeps all the store offsets from being hoisted
  const __amdgpu_buffer_rsrc_t ro = make_rsrc(o.out, (int64_t)o.rows * o.ldo * esz);
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(o.c, ADD ? (int64_t)o.rows * o.ldo * esz : 0);
  const int q = lane >> 4, row = wrow + (lane & 15);
  v4f cscale[NJ];
  float rscale[MI];
  if constexpr (MODE == kInt8) {
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(o.a_scales, (int64_t)o.rows * 4);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(o.b_scales, (int64_t)o.cols * 4);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      cscale[j] = __builtin_bit_cast(
          v4f, __builtin_amdgcn_raw_buffer_load_b128(rb, 4 * (wcol + 16 * j + 4 * q), 0, 0));
#pragma unroll
    for (int i = 0; i < MI; ++i)
      rscale[i] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(ra, 4 * (row + 16 * i), 0, 0));
  }
  Addend<F32> c[2][NJ];
  if constexpr (ADD) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      c[0][j].load(rc, block_off<esz>(ldo, row, wcol + 16 * j + 4 * q, o.cols));
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    if constexpr (ADD) {
      fence();
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (i + 1 < MI)
          c[(i + 1) & 1][j].load(
              rc, block_off<esz>(ldo, row + 16 * (i + 1), wcol + 16 * j + 4 * q, o.cols));
    }
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      fence();
      v4f y0 = acc[i][j], y1 = acc[i][j + 1];
      asm volatile("" : "+v"(y0), "+v"(y1));
      if constexpr (MODE == kInt8) {
        const v4i s0 = __builtin_bit_cast(v4i, y0), s1 = __builtin_bit_cast(v4i, y1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y0[e] = ((float)s0[e] * rscale[i]) * cscale[j][e];
          y1[e] = ((float)s1[e] * rscale[i]) * cscale[j + 1][e];
        }
      }
      if constexpr (ADD) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y0[e] += c[i & 1][j].template at<F16>(e);
          y1[e] += c[i & 1][j + 1].template at<F16>(e);
        }
      }
      store_pair<F32, F16>(y0, y1, ro, ldo, row + 16 * i, wcol + 16 * j, q, o.cols);
      fence();
    }
  }
}

template <int MODE, bool F16, int MI, int NJ>
__device__ __forceinline__ void store_blocks(const v4f (&acc)[MI][NJ], const OutTile& o,
                                             int out_f32, int wrow, int wcol, int lane) {
  if (MODE != kInt8 && o.c != nullptr) {
    if (out_f32) store_rows<MODE, F16, true, true>(acc, o, wrow, wcol, lane);
    else store_rows<MODE, F16, false, true>(acc, o, wrow, wcol, lane);
  } else {
    if (out_f32) store_rows<MODE, F16, true, false>(acc, o, wrow, wcol, lane);
    else store_rows<MODE, F16, false, false>(acc, o, wrow, wcol, lane);
  }
}

// ---------------------------------------------------------------- split contractions

// With T tiles on a grid of P workgroups the last round holds L = T mod P tiles
// (all of them when T < P).  Given a workspace, each of those is split along the
// contraction into S <= min(P / L, kSplitMax) parts of whole stages; place
// S t + s of that round takes part s of its tile t and writes its float32
// accumulators to the workspace, and a second kernel on the same stream adds each
// tile's parts in the order s = 0, 1, .. and stores the tile, so the result does
// not depend on which part ended first.
//
// Workspace: header (L, S), a record for each split tile, then the parts.
constexpr int kSplitMax = 32;
constexpr int kLeastStages = 4;  // of a part
constexpr int64_t kWsHeader = 16384;
constexpr int kMaxSplitTiles = (int)((kWsHeader - 64) / 32);

struct SplitRecord {
  int64_t out_off;
  int32_t rows, cols;
  int64_t row0, col0;  // INT8
};
static_assert(sizeof(SplitRecord) == 32, "records fill the header");

// Parts of a contraction of `stages` stages when `left` tiles are on `grid`
// workgroups; a part keeps at least kLeastStages.
__host__ __device__ __forceinline__ int split_parts(int grid, int left, int stages) {
  if (left <= 0 || left > kMaxSplitTiles) return 1;
#ifdef __HIP_DEVICE_COMPILE__
  int s = div_small(grid, left);
#else
  int s = grid / left;
#endif
  if (s > kSplitMax) s = kSplitMax;
  if (s > stages / kLeastStages) s = stages / kLeastStages;
  return s < 2 ? 1 : s;
}

// The rounds of a launch: `full` whole ones, then `left` tiles in nsplit parts each.
// slot: this workgroup's place in the whole rounds; last_slot: in the last one.  SPREAD
// deals its places, if they are fewer, out over all XCDs: the slots of an XCD are
// consecutive, so that 256 of 512 would lie on four of the eight, twice on each of their
// compute units.  (70 calls of random sizes: 2 % less time in the small form; the large
// one, with one workgroup a compute unit, loses 1 % in shared panels and does without.)
struct Rounds {
  int full, left, nsplit, slot, last_slot;
};

template <int MODE, bool SPREAD>
__device__ __forceinline__ Rounds plan_rounds(const Args& p, int total) {
  Rounds r;
  r.full = div_by(total, p.grid);
  r.left = total - r.full * (int)p.grid.d;
  r.nsplit = 1;
  if (p.ws != nullptr) {
    const int64_t kl = MODE == kWgrad ? p.rows_cap : p.k;
    r.nsplit = split_parts((int)p.grid.d, r.left, (int)((kl + kStageK - 1) / kStageK));
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      int32_t* hdr = reinterpret_cast<int32_t*>(p.ws);
      hdr[0] = r.nsplit > 1 ? r.left : 0;
      hdr[1] = r.nsplit;
    }
  }
  r.slot = xcd_slot();
  r.last_slot = r.slot;
  if constexpr (SPREAD) {
    const int b = (int)blockIdx.x, places = (r.left * r.nsplit + kXcds - 1) / kXcds;
    r.last_slot = b;
    if (places * kXcds <= (int)p.grid.d && b < places * kXcds)
      r.last_slot = b % kXcds * places + b / kXcds;
  }
  return r;
}

struct Work {
  int tile, part, nparts;  // part < 0: a whole tile
  int slot;                // of a part
};

// The work of a workgroup in a round; tile < 0: none left.
__device__ __forceinline__ Work take_work(const Args& p, const Rounds& r, int round) {
  Work k;
  k.part = -1;
  k.nparts = 1;
  k.slot = r.last_slot;
  if (round < r.full) {
    k.tile = round * (int)p.grid.d + r.slot;
  } else if (round > r.full || r.last_slot >= r.left * r.nsplit) {
    k.tile = -1;
  } else if (r.nsplit > 1) {
    const int t = div_small(r.last_slot, r.nsplit);
    k.tile = round * (int)p.grid.d + t;
    k.part = r.last_slot - t * r.nsplit;
    k.nparts = r.nsplit;
  } else {
    k.tile = round * (int)p.grid.d + r.last_slot;
  }
  return k;
}

template <int MODE>
__device__ __forceinline__ void write_split_record(char* ws, int slot, int nsplit, const Tile& t) {
  if (threadIdx.x == 0) {
    SplitRecord* rec = reinterpret_cast<SplitRecord*>(ws + 64) + slot / nsplit;
    rec->out_off = t.out_off;
    rec->rows = t.a_rows;
    rec->cols = t.b_rows;
    if constexpr (MODE == kInt8) {
      rec->row0 = t.row0;
      rec->col0 = t.col0;
    }
  }
}

// Narrows a tile to its part of the contraction.
template <int MODE>
__device__ __forceinline__ void narrow_tile(Tile& t, int part, int nsplit) {
  const int stages = (t.kl + kStageK - 1) / kStageK;
  const int k0 = (int)((int64_t)stages * part / nsplit) * kStageK;
  int k1 = (int)((int64_t)stages * (part + 1) / nsplit) * kStageK;
  if (k1 > t.kl) k1 = t.kl;
  t.a += kColsA<MODE> ? (int64_t)k0 * t.lda : k0;
  t.b += kColsB<MODE> ? (int64_t)k0 * t.ldb : k0;
  t.kl = k1 - k0;
}

// A wave's accumulators as blocks of 256 floats, [lane][4]; rows past the live
// ones are left out.
template <int MI, int NJ>
__device__ __forceinline__ void store_part(float* __restrict__ part, const v4f (&acc)[MI][NJ],
                                           int w, int lane, int wrow, int rows) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      fence();
      v4f y = acc[i][j];
      asm volatile("" : "+v"(y));
      if (wrow + 16 * i + (lane & 15) < rows)
        *reinterpret_cast<v4f*>(part + ((w * MI + i) * NJ + j) * 256 + 4 * lane) = y;
      fence();
    }
}

// The second step of a split: wave by wave one pair of blocks of a split tile.
template <bool I8, bool F16, int BM, int BN, int WN, int MI, int NJ>
__global__ __launch_bounds__(kThreads) void split_reduce_kernel(const char* __restrict__ ws,
                                                                char* out, const char* c,
                                                                int64_t ldo, int out_f32,
                                                                const float* a_scales,
                                                                const float* b_scales) {
  constexpr int kUnits = BM * BN / 512;
  const int32_t* hdr = reinterpret_cast<const int32_t*>(ws);
  const int nl = hdr[0], nsplit = hdr[1];
  if (nl <= 0) return;
  const SplitRecord* recs = reinterpret_cast<const SplitRecord*>(ws + 64);
  const float* parts = reinterpret_cast<const float*>(ws + kWsHeader);
  const int lane = threadIdx.x & 63;
  const int stride = (int)gridDim.x * (kThreads / 64);
  for (int it = uni((int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6)); it < nl * kUnits;
       it += stride) {
    const int l = it / kUnits, u = it % kUnits;
    const int w = u / (MI * NJ / 2), i = u / (NJ / 2) % MI, j = u % (NJ / 2) * 2;
    const SplitRecord rec = recs[l];
    const int wrow = (w / WN) * (16 * MI) + 16 * i, wcol = (w % WN) * (16 * NJ) + 16 * j;
    if (wrow >= rec.rows || wcol >= rec.cols) continue;
    v4f y[1][2];
    y[0][0] = y[0][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (wrow + (lane & 15) < rec.rows) {
      const float* src = parts + (int64_t)l * nsplit * (BM * BN) + u * 512 + 4 * lane;
#pragma unroll 8
      for (int s = 0; s < nsplit; ++s) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const v4f v = *reinterpret_cast<const v4f*>(src + (int64_t)s * (BM * BN) + 256 * b);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (I8)
              y[0][b][e] = __int_as_float(__float_as_int(y[0][b][e]) + __float_as_int(v[e]));
            else
              y[0][b][e] += v[e];
          }
        }
      }
    }
    OutTile o;
    o.out = out + rec.out_off;
    o.c = c != nullptr ? c + rec.out_off : nullptr;
    o.ldo = (int)ldo;
    o.rows = rec.rows;
    o.cols = rec.cols;
    o.a_scales = I8 ? a_scales + rec.row0 : nullptr;
    o.b_scales = I8 ? b_scales + rec.col0 : nullptr;
    store_blocks<I8 ? kInt8 : kFprop, F16, 1, 2>(y, o, out_f32, wrow, wcol, lane);
  }
}

// Workgroups of the second step: at most half of the slots hold split tiles.
inline unsigned reduce_grid(int slots, int units) {
  const int64_t waves = (int64_t)(slots / 2) * units, cap = 8 * (int64_t)device_cu_count();
  const int64_t wgs = (waves + kThreads / 64 - 1) / (kThreads / 64);
  return (unsigned)(wgs < cap ? wgs : cap);
}

// Grid of a launch with `slots` workgroups resident (0: nothing to do), and the numbers
// that the kernel divides by.  Where the host knows that no tile is split it leaves the
// workspace out, and the second step is not launched: contractions too short for two
// parts, and weight gradients (whose tiles it can count) whose rounds come out even.
template <int MODE, int BM, int BN>
int prepare_launch(Args& p, int slots) {
  const int64_t ntn = ((MODE == kWgrad ? p.k : p.n) + BN - 1) / BN;
  const int64_t bound =
      MODE == kWgrad ? p.G * ((p.n + BM - 1) / BM) * ntn
                     : ((p.rows_cap + BM - 1) / BM + (MODE == kLora ? 0 : p.G)) * ntn;
  const int stages = (int)(((MODE == kWgrad ? p.rows_cap : p.k) + kStageK - 1) / kStageK);
  const int most = p.ws != nullptr ? split_parts(slots, 1, stages) : 1;
  const int grid = (int)(bound * most < slots ? bound * most : slots);
  if (grid <= 0) return 0;
  if (most < 2 || (MODE == kWgrad && split_parts(grid, (int)(bound % grid), stages) < 2))
    p.ws = nullptr;
  p.grid = make_div(grid);
  p.band = make_div(kSuperM * ntn);
  return grid;
}

template <int MODE>
__device__ __forceinline__ OutTile out_tile(const Args& p, const Tile& t) {
  OutTile o;
  o.out = p.out + t.out_off;
  o.c = p.c != nullptr ? p.c + t.out_off : nullptr;
  o.ldo = (int)p.ldo;
  o.rows = t.a_rows;
  o.cols = t.b_rows;
  o.a_scales = MODE == kInt8 ? p.a_scales + t.row0 : nullptr;
  o.b_scales = MODE == kInt8 ? p.b_scales + t.col0 : nullptr;
  return o;
}

// ---------------------------------------------------------------- launchers

hipError_t launch_large(int mode, int f16, const Args& p, hipStream_t stream);
hipError_t launch_small(int mode, int f16, int bm, const Args& p, hipStream_t stream);
hipError_t launch_large_int8(int f16, const Args& p, hipStream_t stream);
hipError_t launch_small_int8(int f16, int bm, const Args& p, hipStream_t stream);
size_t large_workspace_bytes();
size_t small_workspace_bytes();

// Rows of the tiles of the form that a call takes.
int form_rows(int mode, int64_t G, int64_t rows_cap, int64_t n, int64_t k, bool split);

}  // namespace g16
}  // namespace bsg

#endif  // BSG_GEMM_16BIT_H
