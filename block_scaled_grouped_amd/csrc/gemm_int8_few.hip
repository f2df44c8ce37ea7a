// Products of 8-bit integers for few rows (a decoding step): the weights' bytes bound them.
//
// A tile is 16 columns of a group's weights and up to 16 of its rows; a workgroup takes one
// after the other.  Its waves share out the contraction in lines of 128 bytes and add their
// sums through LDS.  Every wave copies its own lines global -> LDS into a ring of its own,
// whole lines at a time and on into the next tile, and waits for nobody else's; from there
// they go to the matrix instruction (v_mfma_i32_16x16x64: lane (r, q) = (l % 16, l / 16)
// holds 16 bytes of column r).  Loaded straight into the registers, 16 neighbouring lanes ask
// for 16 lines: 64 rows of 41 experts x 2048 x 7168 took 143 us, a tile at a time through the
// ring 118, and now 107 (5.6 TB/s).  One row x 14336 x 4096 in 16-bit tokens takes 11.9 us
// from call to call (58.8 MB at 4.9 TB/s), 15.6 with a launch for the tokens, 20.5 with that
// and split 32-row tiles.
//
// TOKENS: the rows are in 16 bits.  Every workgroup quantizes the rows itself, into LDS, while
// its first weights are on their way: one launch instead of two, for calls of so few rows
// that this costs less than the launch.  Else they are integers and come through the ring too.
#include "bsg_internal.h"
#include "lds_dma.h"
#include "quantize_row.h"

namespace bsg {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 16;      // of a tile
constexpr int kLine = 128;     // bytes of the contraction a wave takes at a time
constexpr int kSlots = 3;      // of a wave's ring: lines in flight (2 % better than 4)
constexpr int kBlock = kRows * kLine;  // bytes of 16 rows' lines
constexpr int kPad = 16;       // between rows in LDS, so that 16 lanes' reads meet no bank twice

struct Args {
  const void* x;       // [rows_cap, k]: 16-bit tokens, or integers
  const float* a_scales;
  int64_t ldx;         // elements
  const int8_t* b;
  const float* b_scales;
  const int64_t* offsets;
  char* out;
  int64_t ldb, stride_b, ldo, rows_cap;
  uint32_t* status;
  int G, n, k, f16, out_f32;
  int rows_held;       // TOKENS: rows that LDS has room for
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uni64(int64_t v) {
  const uint32_t lo = (uint32_t)uni((int)(v & 0xffffffff)), hi = (uint32_t)uni((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ uint32_t lds_of(const int8_t* shared_ptr) {
  return (uint32_t)(size_t)(__attribute__((address_space(3))) const int8_t*)shared_ptr;
}

// A lane's share of the copies of 16 rows' lines: rows 8 p + l / 8, p = 0 and 1, the chunk
// of 16 bytes that belongs in slot l % 8 of the row.  Chunk c of row r lies in slot
// c ^ ((r / 2) % 8), so that 16 lanes reading a chunk of 16 rows hit all 64 banks.
struct Lines {
  int row[2], chunk[2];
  __device__ __forceinline__ void init(int rows, int64_t ld, int lane) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 8 * p + (lane >> 3);
      row[p] = r < rows ? r * (int)ld : kDmaOutOfRange;
      chunk[p] = 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
  }
  // at: byte of the contraction that the line begins with.  Past the contraction or the rows:
  // zeros
  __device__ __forceinline__ void copy(const v4i& rsrc, uint32_t lds, int at, int k) const {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int e = at + chunk[p];
      dma16(rsrc, lds + 1024 * p, e < k && row[p] != kDmaOutOfRange ? row[p] + e : kDmaOutOfRange);
    }
  }
};

// Where a tile lies.
struct Tile {
  int64_t row0;
  int g, nt, rows;
};

template <bool TOKENS, bool F16>
__global__ __launch_bounds__(kThreads) void few_rows_kernel(Args p) {
  constexpr int kSlotBytes = TOKENS ? kBlock : 2 * kBlock;  // weights, then rows
  constexpr int kCopies = kSlotBytes / 1024;
  __shared__ __attribute__((aligned(16))) int8_t ring[kWaves][kSlots * kSlotBytes];
  // TOKENS: the rows as they are, in whole pieces of 1 KiB, then their integers [rows][k + kPad]
  extern __shared__ __attribute__((aligned(16))) int8_t tokens[];
  __shared__ v4i sums[2][kWaves][64];
  __shared__ int64_t off[kMaxGroups + 1];
  __shared__ int32_t cnt[kMaxGroups], pre[kMaxGroups + 1];
  __shared__ float scales[kRows];
  __shared__ uint32_t peak[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int ntn = (p.n + 15) / 16, k = p.k;
  const int lines = (k + kLine - 1) / kLine, pitch = k + kPad;
  const int mine = (lines - w + kWaves - 1) / kWaves;  // this wave's lines: w, w + kWaves, ..
  const uint32_t lds = (uint32_t)(size_t)(__attribute__((address_space(3))) int8_t*)ring[w];
  int64_t first = 0, count = 0;  // one group: its rows
  int total;
  if (p.G == 1) {
    first = p.offsets[0];
    int64_t last = p.offsets[1];
    const uint32_t bad = (first < 0 || last < first ? kDevNegativeSize : 0u) |
                         (first > p.rows_cap || last > p.rows_cap ? kDevOverCapacity : 0u);
    if (bad != 0 && blockIdx.x == 0 && tid == 0) dev_status_or(p.status, bad);
    first = first < 0 ? 0 : first > p.rows_cap ? p.rows_cap : first;
    last = last < 0 ? 0 : last > p.rows_cap ? p.rows_cap : last;
    first = uni64(first);
    count = uni64(last > first ? last - first : 0);
    total = (int)((count + kRows - 1) / kRows) * ntn;
  } else {
    load_offsets_clamped(p.offsets, p.G, p.rows_cap, off, blockIdx.x == 0 ? p.status : nullptr);
    for (int g = tid; g < p.G; g += kThreads)
      cnt[g] = (int32_t)((group_extent(off, g) + kRows - 1) / kRows) * ntn;
    __syncthreads();
    wave0_exclusive_scan(cnt, p.G, pre);
    __syncthreads();
    total = uni(pre[p.G]);
  }
  const auto locate = [&](int tile) {
    Tile t;
    int u = tile;
    int64_t begin = first, extent = count;
    t.g = 0;
    if (p.G > 1) {
      t.g = uni(find_group(pre, p.G, tile));
      u -= uni(pre[t.g]);
      begin = uni64(off[t.g]);
      extent = uni64(group_extent(off, t.g));
    }
    // blocks of rows innermost: neighbours in the order run on one XCD and share the weights
    const int mtiles = (int)((extent + kRows - 1) / kRows);
    t.nt = mtiles > 1 ? u / mtiles : u;
    const int mt = u - t.nt * mtiles;
    t.row0 = begin + (int64_t)mt * kRows;
    const int64_t left = extent - (int64_t)mt * kRows;
    t.rows = uni((int)(left < kRows ? left : kRows));
    return t;
  };

  // The copies run kSlots lines ahead, through all of the workgroup's tiles.
  Lines lb, la;
  int to_tile = xcd_slot(), to_line = 0, to_slot = 0;
  int64_t b_base = 0, a_base = 0;
  int b_bytes = 0, a_bytes = 0;
  const auto aim = [&]() {
    b_bytes = a_bytes = 0;  // past the last tile: zeros
    if (to_tile < total) {
      const Tile t = locate(to_tile);
      const int cols = uni(p.n - 16 * t.nt < 16 ? p.n - 16 * t.nt : 16);
      b_base = (int64_t)(p.b + t.g * p.stride_b + (int64_t)(16 * t.nt) * p.ldb);
      b_bytes = (cols - 1) * (int)p.ldb + k;
      lb.init(cols, p.ldb, lane);
      if constexpr (!TOKENS) {
        a_base = (int64_t)(static_cast<const int8_t*>(p.x) + t.row0 * p.ldx);
        a_bytes = (t.rows - 1) * (int)p.ldx + k;
        la.init(t.rows, p.ldx, lane);
      }
    }
  };
  const auto copy_next = [&]() {
    const uint32_t at = lds + to_slot * kSlotBytes;
    const int e = (w + kWaves * to_line) * kLine;
    lb.copy(make_rsrc_words(reinterpret_cast<const void*>(b_base), b_bytes), at, e, k);
    if constexpr (!TOKENS)
      la.copy(make_rsrc_words(reinterpret_cast<const void*>(a_base), a_bytes), at + kBlock, e, k);
    to_slot = to_slot + 1 == kSlots ? 0 : to_slot + 1;
    if (++to_line >= mine) {
      to_line = 0;
      to_tile += (int)gridDim.x;
      aim();
    }
  };
  lb.init(1, p.ldb, lane);
  if constexpr (!TOKENS) la.init(1, p.ldx, lane);

  int tile = xcd_slot(), slot = 0;
  if (tile >= total) return;
  int64_t held = -1;  // TOKENS: first of the rows that are in LDS, and how many
  int held_rows = 0;
  const int pieces = (2 * k + 1023) / 1024;  // of a row
  int8_t* const codes = tokens + (TOKENS ? p.rows_held : 0) * pieces * 1024;
  // Copies the tile's rows as they are.
  const auto copy_tokens = [&](const Tile& t) {
    for (int row = 0; row < t.rows; ++row) {
      const v4i rs = make_rsrc_words(static_cast<const uint16_t*>(p.x) + (t.row0 + row) * p.ldx,
                                     2 * k);
      for (int i = w; i < pieces; i += kWaves)
        dma16(rs, lds_of(tokens) + (row * pieces + i) * 1024, i * 1024 + 16 * lane);
    }
  };
  const auto quantize_tokens = [&](const Tile& t) {
    // 256, 128 or 64 threads a row
    const int per = t.rows > 2 ? 4 : t.rows > 1 ? 2 : 1, threads = kThreads / per;
    const int sub = tid / threads, i = tid % threads;
    for (int r0 = 0; r0 < t.rows; r0 += per) {
      const int row = r0 + sub;
      const bool here = row < t.rows;
      const int8_t* src = tokens + (here ? row : 0) * pieces * 1024;
      uint32_t m = 0;
      for (int e = 8 * i; e < k; e += 8 * threads)
        m = max_magnitude(m, *reinterpret_cast<const v4i*>(src + 2 * e));
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
      if (lane == 0) peak[w] = m;
      __syncthreads();
      for (int v = 0; v < threads / 64; ++v) m = max(m, peak[sub * (threads / 64) + v]);
      bool finite;
      const RowScale s = row_scale<F16>(m, finite);
      if (here) {
        if (i == 0) {
          scales[row] = s.s;
          if (!finite && t.nt == 0) dev_status_or(p.status, kDevNonFinite);
        }
        for (int e = 8 * i; e < k; e += 8 * threads)
          *reinterpret_cast<v2i*>(codes + row * pitch + e) =
              quantize8<F16>(*reinterpret_cast<const v4i*>(src + 2 * e), s, finite);
      }
      __syncthreads();
    }
  };

  Tile t = locate(tile);
  if constexpr (TOKENS) copy_tokens(t);
  aim();
  if (mine > 0) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) copy_next();
  }
  for (int turn = 0;; ++turn) {
    if constexpr (TOKENS) {
      if (t.row0 != held || t.rows != held_rows) {
        if (held < 0) {  // the copies of the first weights came after the rows'
          asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kSlots * kCopies) : "memory");
          if (mine == 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        } else {
          __syncthreads();  // the rows before have been read
          copy_tokens(t);
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        __syncthreads();
        quantize_tokens(t);
        held = t.row0;
        held_rows = t.rows;
      }
    }
    // rows past the last repeat it: what they give is not stored
    const int8_t* arow = codes + (r < t.rows ? r : t.rows - 1) * pitch;
    v4i acc = v4i{0, 0, 0, 0};
    for (int i = 0; i < mine; ++i) {
      // this wave's copies complete in order: the line's have landed, later ones need not
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kSlots - 1) * kCopies) : "memory");
      const int8_t* from = ring[w] + slot * kSlotBytes + r * kLine;
      slot = slot + 1 == kSlots ? 0 : slot + 1;
      v4i bv[2], av[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = 4 * h + q, at = (w + kWaves * i) * kLine + 16 * c;
        const int place = (c ^ ((r >> 1) & 7)) << 4;
        bv[h] = *reinterpret_cast<const v4i*>(from + place);
        if constexpr (TOKENS) av[h] = *reinterpret_cast<const v4i*>(arow + (at < k ? at : 0));
        else av[h] = *reinterpret_cast<const v4i*>(from + kBlock + place);
      }
      // the slot has been read before it is copied to again
      asm volatile("s_waitcnt lgkmcnt(0)"
                   : "+v"(bv[0]), "+v"(bv[1]), "+v"(av[0]), "+v"(av[1])
                   :
                   : "memory");
      copy_next();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[h], av[h], acc, 0, 0, 0);
    }
    sums[turn & 1][w][lane] = acc;
    // the waves take turns at the tiles' ends, so two sets of sums and one barrier do
    __syncthreads();
    if (w == (turn & (kWaves - 1))) {
      v4i s = sums[turn & 1][0][lane];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) {
        const v4i o = sums[turn & 1][i][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += o[e];
      }
      const int col = 16 * t.nt + 4 * q;
      if (r < t.rows && col < p.n) {
        const v4f bs = *reinterpret_cast<const v4f*>(p.b_scales + (int64_t)t.g * p.n + col);
        const float as = TOKENS ? scales[r] : p.a_scales[t.row0 + r];
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = ((float)s[e] * as) * bs[e];
        const int64_t at = (t.row0 + r) * p.ldo + col;
        if (p.out_f32)
          *reinterpret_cast<v4f*>(p.out + 4 * at) = v4f{y[0], y[1], y[2], y[3]};
        else if (p.f16)
          *reinterpret_cast<v2i*>(p.out + 2 * at) =
              v2i{(int)pack16<true>(y[0], y[1]), (int)pack16<true>(y[2], y[3])};
        else
          *reinterpret_cast<v2i*>(p.out + 2 * at) =
              v2i{(int)pack16<false>(y[0], y[1]), (int)pack16<false>(y[2], y[3])};
      }
    }
    tile += (int)gridDim.x;
    if (tile >= total) break;
    t = locate(tile);
  }
  // no copy is in flight when the workgroup's LDS goes to another
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Workgroups: all tiles that there can be, as many to each, two workgroups a compute unit at
// most (32 KiB of weights on their way to one are enough).
unsigned grid_for(int64_t G, int64_t rows_cap, int64_t n) {
  // nonempty groups and 16 rows more make a block of rows
  const int64_t groups = rows_cap < G ? rows_cap : G;
  const int64_t blocks = groups + (rows_cap - groups) / kRows;
  const int64_t tiles = blocks * ((n + 15) / 16), cap = 2 * (int64_t)device_cu_count();
  const int64_t rounds = (tiles + cap - 1) / cap;
  const int64_t grid = ((tiles + rounds - 1) / rounds + kXcds - 1) / kXcds * kXcds;
  return (unsigned)(grid < tiles ? grid : tiles);
}

}  // namespace

hipError_t launch_gemm_int8_few(int tokens, int in_f16, int G, const void* x, int64_t ldx,
                                const float* a_scales, const int8_t* b, int64_t ldb,
                                int64_t stride_b, const float* b_scales, const int64_t* offsets,
                                int64_t rows_cap, int64_t n, int64_t k, void* out, int64_t ldo,
                                int f16, int out_f32, uint32_t* status, hipStream_t stream) {
  if (rows_cap == 0) return hipSuccess;
  const int64_t rows = rows_cap < kRows ? rows_cap : kRows;
  const Args p{x, a_scales, ldx, b, b_scales, offsets, static_cast<char*>(out), ldb, stride_b, ldo,
               rows_cap, status, G, (int)n, (int)k, f16, out_f32, (int)rows};
  const unsigned lds = tokens ? (unsigned)(rows * ((2 * k + 1023) / 1024 * 1024 + k + kPad)) : 0;
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid_for(G, rows_cap, n)), dim3(kThreads), lds, stream, p);
    return hipGetLastError();
  };
  if (!tokens) return run(few_rows_kernel<false, false>);
  return in_f16 ? run(few_rows_kernel<true, true>)
                : run(few_rows_kernel<true, false>);
}

}  // namespace bsg
