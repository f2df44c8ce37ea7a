// The router of a mixture of experts: each token's top k experts, their weights, the
// tokens of each expert and a loss that balances them; and the gradient of the logits.
//
// With l the logits of a token that is routed (live), n the live tokens:
//   p_e = exp(l_e - max l) / sum_i exp(l_i - max l)
//   the k largest logits, ties to the lowest index; -inf and NaN are never chosen
//   w_j = p_{e_j}, or, normalized, p_{e_j} / sum_i p_{e_i}
//   c_e = how often e is chosen, S_e = sum of p_e over the live tokens
//   loss = E / (k n^2) * sum_e c_e S_e
// and backwards, with b_e = dloss * E c_e / (k n^2) (the counts are constants):
//   unnormalized  a_e = b_e + sum_j dw_j [e_j = e],  dl_e = p_e (a_e - sum_i p_i a_i)
//   normalized    dl_e = p_e (b_e - sum_i p_i b_i) + sum_j [e_j = e] w_j (dw_j - sum_i w_i dw_i)
//
// 16 lanes take a token, EPL experts each, so that a wave holds four tokens and reductions
// are lane moves within a row of 16 (DPP).  A lane's experts are runs of 16 bytes, 16 lanes
// apart: a load of the wave covers whole lines of its four rows.
//
// The largest are found on 32-bit keys: the logit's bits, ordered as integers, with the
// lowest eight replaced by 255 - index.  Keys differ, so the next largest below M is the
// one with the largest key - M (unsigned: those at or above M come out smallest), which
// takes a subtraction and half a three-way maximum each, and no search for an index.
// Only the differences compare so: M is added back after the maximum over the lanes, for
// a lane with nothing below M would come out with a key at or above it.
// A 16-bit logit has its bits above those eight.  A float32 one may share them with the
// next in order: where that happens among a token's k + 1 largest the wave does it again,
// on whole values.
//
// What bounds it: the forward pass the vector units (busy 0.76 of the time; 550 instructions for a
// wave's four tokens of 256 experts), the backward pass HBM.  65536 float32 tokens of 256 experts,
// k 8: forward 25 us (67 MB; some 3 of them until the first tokens are there), adding up 4.7,
// backward 27.7 (139 MB at 5.0 TB/s).  16384 bf16 tokens of 64 experts 5.9, 4.6 to 5.0 and 5.7; 64 of
// 8 3.6 in one launch.  Two workgroups a compute unit (forward) are slower: 35 us.  Float32 tokens of
// 129 to 256 experts in runs of one take all 128 registers and spill five more (forward, the only
// form that does).
#include <type_traits>

#include "bsg_internal.h"

namespace bsg {

namespace {

constexpr int kLanes = 16;           // of a token
constexpr int kMaxExperts = 256;
constexpr int kFwdThreads = 1024;
constexpr int kFwdTokens = kFwdThreads / kLanes;
constexpr int kFwdWaves = kFwdThreads / 64;
constexpr int kFwdBlocks = 256;      // at most: one a compute unit
constexpr int64_t kOneBlock = 256;   // tokens that one workgroup takes alone
constexpr int kBwdThreads = 256;
constexpr int kBwdTokens = kBwdThreads / kLanes;

typedef __attribute__((address_space(1))) const char gchar;

// ---------------------------------------------------------------- 16 lanes

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// f over the 16 lanes, the same bits in all of them: f is commutative.
template <typename F>
__device__ __forceinline__ uint32_t reduce16(uint32_t v, F f) {
  v = f(v, dpp<kXor1>(v));
  v = f(v, dpp<kXor2>(v));
  v = f(v, dpp<kHalfMirror>(v));
  return f(v, dpp<kMirror>(v));
}
__device__ __forceinline__ uint32_t max16u(uint32_t v) {
  return reduce16(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t min16u(uint32_t v) {
  return reduce16(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ float max16(float v) {
  return __uint_as_float(reduce16(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float sum16(float v) {
  return __uint_as_float(reduce16(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// ---------------------------------------------------------------- values

// exp(x) for x <= 0 or NaN: the product's rounding is |x| 2^-24 of the result.
__device__ __forceinline__ float exp_le0(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269502162933349609375f);
}

// DT 0: bf16, 1: fp16, 2: float32.
template <int DT> constexpr int kBytes = DT == 2 ? 4 : 2;
template <int DT>
__device__ __forceinline__ float decode16(uint32_t bits) {
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  return __uint_as_float(bits << 16);
}
// A lane's experts: runs of kRun, a run of the 16 lanes after the other.  RUNS: the experts are
// whole runs of 16 bytes (or what a lane has); else runs of one, which neighbouring lanes load and
// store next to each other (65536 x 250 float32: forward 36 and backward 49 us with runs of four
// taken one by one, now 26 and 27).
template <int DT, int EPL, bool RUNS>
constexpr int kRun = !RUNS ? 1 : EPL < 16 / kBytes<DT> ? EPL : 16 / kBytes<DT>;
template <int DT, int EPL, bool RUNS>
__device__ __forceinline__ int expert_of(int slot, int j) {
  constexpr int R = kRun<DT, EPL, RUNS>;
  return R * (slot + kLanes * (j / R)) + j % R;
}

// A row is aligned to its elements only; the hardware takes wide loads and stores at any.
typedef v4i v4i_any __attribute__((aligned(2)));
typedef v2i v2i_any __attribute__((aligned(2)));
typedef int int_any __attribute__((aligned(2)));
#define BSG_GLOBAL __attribute__((address_space(1)))

// A lane's logits; those past the last expert are anything.
template <int DT, int EPL, bool RUNS>
__device__ __forceinline__ void load_row(const char* row, int slot, int E, float (&v)[EPL]) {
  constexpr int R = kRun<DT, EPL, RUNS>, bytes = R * kBytes<DT>;
#pragma unroll
  for (int c = 0; c < EPL / R; ++c) {
    const int e0 = R * (slot + kLanes * c);
    float* out = v + R * c;
    uint32_t w[(bytes + 3) / 4];
    const gchar* at = (const gchar*)(row) + (int64_t)(e0 < E ? e0 : 0) * kBytes<DT>;
    if constexpr (bytes == 16) {
      const v4i q = *reinterpret_cast<const BSG_GLOBAL v4i_any*>(at);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (uint32_t)q[j];
    } else if constexpr (bytes == 8) {
      const v2i q = *reinterpret_cast<const BSG_GLOBAL v2i_any*>(at);
      w[0] = (uint32_t)q[0];
      w[1] = (uint32_t)q[1];
    } else if constexpr (bytes == 4) {
      w[0] = (uint32_t)*reinterpret_cast<const BSG_GLOBAL int_any*>(at);
    } else {
      w[0] = *reinterpret_cast<const BSG_GLOBAL uint16_t*>(at);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if constexpr (DT == 2) out[j] = __uint_as_float(w[j]);
      else out[j] = decode16<DT>((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
    }
  }
}

// -inf for experts that are not there, and all of a token that is not to be routed.  Nothing to
// do, for the whole wave, where its tokens are routed and the experts fill their lanes.
template <int DT, int EPL, bool RUNS>
__device__ __forceinline__ void close_absent(float (&v)[EPL], bool routed, int slot, int E) {
  if (E == kLanes * EPL && __all(routed)) return;
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    v[j] = routed && expert_of<DT, EPL, RUNS>(slot, j) < E ? v[j] : -INFINITY;
}

template <int DT, int EPL, bool RUNS>
__device__ __forceinline__ void store_row(char* row, int slot, int E, const float (&v)[EPL]) {
  constexpr int R = kRun<DT, EPL, RUNS>, bytes = R * kBytes<DT>, words = (bytes + 3) / 4;
#pragma unroll
  for (int c = 0; c < EPL / R; ++c) {
    const int e0 = R * (slot + kLanes * c);
    const float* in = v + R * c;
    uint32_t w[words];
#pragma unroll
    for (int j = 0; j < words; ++j) {
      if constexpr (DT == 2) w[j] = __float_as_uint(in[j]);
      else w[j] = pack16<DT == 1>(in[2 * j], R > 1 ? in[(2 * j + 1) % R] : 0.0f);
    }
    BSG_GLOBAL char* at = (BSG_GLOBAL char*)(row) + (int64_t)e0 * kBytes<DT>;
    if (e0 >= E) continue;
    if constexpr (bytes == 16)
      *reinterpret_cast<BSG_GLOBAL v4i_any*>(at) = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    else if constexpr (bytes == 8)
      *reinterpret_cast<BSG_GLOBAL v2i_any*>(at) = v2i{(int)w[0], (int)w[1]};
    else if constexpr (bytes == 4)
      *reinterpret_cast<BSG_GLOBAL int_any*>(at) = (int)w[0];
    else
      *reinterpret_cast<BSG_GLOBAL uint16_t*>(at) = (uint16_t)w[0];
  }
}

// A logit's bits ordered as unsigned integers, -0 as 0; not a NaN's.  What is below kOpen is
// not to be chosen.
constexpr uint32_t kOpen = 0x00800000u;  // of the lowest finite number
__device__ __forceinline__ uint32_t order(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// by comparison: of a signalling NaN a maximum of three is a NaN
__device__ __forceinline__ float closed_if_nan(float v) { return v == v ? v : -INFINITY; }

// The middle one of a >= b and x: where x goes among them, b or what b makes room for.
__device__ __forceinline__ uint32_t middle(uint32_t a, uint32_t b, uint32_t x) {
  uint32_t m;
  asm("v_med3_u32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(x));
  return m;
}

template <int N>
__device__ __forceinline__ uint32_t max_of(const uint32_t (&v)[N]) {
  uint32_t m = v[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = m > v[j] ? m : v[j];
  return m;
}

// This lane's of a token's k chosen experts (lane j: the j-th; -1: none).
//
// A round takes the largest of the token's keys.  Each lane holds its own kHeads largest in
// order, so that a round is a maximum over 16 lanes and a step of the winner's list.  A lane
// that used up its list before the last round may have missed a key: of 256 experts' 9
// largest that happens to 2 % of the tokens, and all rounds are done again on all keys (as
// they are at once where more than kFewRounds are asked for).
constexpr int kHeads = 4, kFewRounds = 9, kRoundsAtOnce = 3;

// key: of the lane's experts.  whole(key) gives them without the index, for float32.
template <int DT, int EPL, bool RUNS, typename F>
__device__ __forceinline__ int choose(uint32_t (&key)[EPL], int slot, int E, int k, F whole) {
  constexpr int H = EPL < kHeads ? EPL : kHeads;
  // float32: one more than is chosen, which shows whether the last is next to another
  const int rounds = DT == 2 && k < E ? k + 1 : k;
  uint32_t mine = 0, m = 0;
  const auto below = [&](uint32_t top) {  // the token's largest key below `top`
    uint32_t d[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) d[j] = key[j] - top;
    return max16u(max_of(d)) + top;
  };
  bool all = EPL > H && rounds > kFewRounds;
  if (!all) {
    uint32_t head[H];
    bool won = false;
    // a key at a time into its place among the largest so far
    head[0] = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) {
      const uint32_t x = key[j];
      if (j < H) head[j % H] = head[j - 1] < x ? head[j - 1] : x;
#pragma unroll
      for (int i = H - 1; i > 0; --i)
        if (i < j) head[i] = middle(head[i - 1], head[i], x);
      head[0] = head[0] > x ? head[0] : x;
    }
    for (int r0 = 0; r0 < rounds; r0 += kRoundsAtOnce) {
#pragma unroll
      for (int r = 0; r < kRoundsAtOnce; ++r) {
        if (r0 + r == rounds) break;
        m = max16u(head[0]);
        mine = slot == r0 + r ? m : mine;
        won = head[0] == m;
#pragma unroll
        for (int i = 0; i < H; ++i) head[i] = won ? (i + 1 < H ? head[(i + 1) % H] : 0u) : head[i];
      }
    }
    all = EPL > H && __any(head[0] == 0 && !won);
  }
  if (EPL > H && all) {
    m = max16u(max_of(key));
    mine = m;
    for (int r = 1; r < rounds; ++r) {
      m = below(m);
      mine = slot == r ? m : mine;
    }
  }
  int chosen = slot < k && mine >= kOpen ? 255 - (int)(mine & 255u) : -1;
  if constexpr (DT == 2) {
    // neighbours in the order, the last round's (in m) next to lane k - 1's
    const uint32_t after = dpp<0x101>(mine);  // of lane + 1, which has to be active
    const uint32_t next = slot == k - 1 ? (rounds > k ? m : 0u) : after;
    if (__any(slot < k && next >= kOpen && (next ^ mine) < 256u)) {
      whole(key);
      chosen = -1;
      for (int r = 0; r < k; ++r) {
        m = max16u(max_of(key));
        uint32_t at = 0xffffu;
#pragma unroll
        for (int j = EPL - 1; j >= 0; --j)
          at = key[j] == m ? (uint32_t)expert_of<DT, EPL, RUNS>(slot, j) : at;
        at = min16u(at);
        if (slot == r && m >= kOpen) chosen = (int)at;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
          key[j] = (uint32_t)expert_of<DT, EPL, RUNS>(slot, j) == at ? 0u : key[j];
      }
    }
  }
  return chosen;
}

// The largest, of numbers.  A NaN may come out as one (it makes the sum NaN in any case).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  return m;
}

// A token's softmax: exp(l - max) in ex, what they have to be multiplied by, and whether it is
// live.  Without an open expert the sum of the exponentials is 0 (max stands for 0 then), with
// a NaN or +inf it is NaN: close_if_all_nan has to follow where a wave has such a token.
struct Softmax {
  float max, sum, inv;
  bool live;
};
template <int EPL>
__device__ __forceinline__ Softmax softmax(const float (&v)[EPL], float (&ex)[EPL]) {
  Softmax r;
  float m = v[0];
#pragma unroll
  for (int j = 1; j < EPL; j += 2) m = max3(m, v[j], v[j + 1 < EPL ? j + 1 : j]);
  // a lane move may not follow what it reads by less than two wait states
  if constexpr (EPL > 1) asm volatile("s_nop 1" : "+v"(m));
  m = max16(m);
  r.max = m > -INFINITY ? m : 0.0f;
  r.sum = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    ex[j] = exp_le0(v[j] - r.max);
    r.sum += ex[j];
  }
  r.sum = sum16(r.sum);
  r.live = !(r.sum == 0.0f);
  r.inv = r.live ? 1.0f / r.sum : 0.0f;
  return r;
}

// A token with a NaN and no open expert is not live: ex is 0, and only the sum tells of the NaN.
template <int EPL>
__device__ __forceinline__ void close_if_all_nan(const float (&v)[EPL], float (&ex)[EPL],
                                                 Softmax& r) {
  float open = -INFINITY;
#pragma unroll
  for (int j = 0; j < EPL; ++j) open = fmaxf(open, closed_if_nan(v[j]));
  if (max16(open) > -INFINITY || r.sum == 0.0f) return;
  r.live = false;
  r.inv = 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) ex[j] = 0.0f;
}

// ---------------------------------------------------------------- forward

struct Fwd {
  const char* logits;
  int64_t ld, tokens;  // ld in bytes
  const uint8_t* mask;
  int E, k, normalize;
  int32_t* experts;
  float* weights;
  int32_t* counts;
  float* prob_sums;
  int32_t* live;
  float* loss;
  uint32_t* status;
  // workspace: of each workgroup (S_e, c_e) [E] and its live tokens; then for the
  // second kernel c_e S_e [E] and a count of its workgroups
  v2i* parts;
  int32_t* part_live;
  double* products;
  uint32_t* done;
};

// Sum over lanes of a wave, in one order.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// loss from sum_e c_e S_e
__device__ __forceinline__ float balance_loss(double products, int E, int k, int live) {
  if (live == 0) return 0.0f;
  return (float)(products * E / ((double)k * live * live));
}

// Orders a wave's LDS accesses before and after (they complete in that order by themselves).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Every workgroup takes 64 tokens at a time, and reads the next 64 ahead; what it sums over
// tokens stays in registers (a lane's experts are the same for all of its tokens) and is
// added up in one order at the end.  Alone, it writes the results itself.
template <int DT, int EPL, bool RUNS>
__global__ __launch_bounds__(kFwdThreads) void router_kernel(Fwd p) {
  // exponentials of the tokens at hand; at the end the waves' sums
  __shared__ __attribute__((aligned(16))) float rows[kFwdTokens][kLanes * EPL];
  float(*sums)[kLanes * EPL] = rows;
  __shared__ int32_t hist[kMaxExperts];
  __shared__ int32_t live_of[kFwdWaves];
  __shared__ double products[kMaxExperts / 64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int slot = lane & (kLanes - 1);
  const int E = p.E, k = p.k;
  if (tid < kMaxExperts) hist[tid] = 0;
  if (blockIdx.x == 0 && tid == 0) *p.done = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) acc[j] = 0.0f;
  int live_tokens = 0;
  bool bad = false;
  float* mine = rows[tid >> 4];
  const int64_t stride = (int64_t)gridDim.x * kFwdTokens;
  int64_t t = (int64_t)blockIdx.x * kFwdTokens + (tid >> 4);
  float v[EPL];
  bool routed;
  const auto load = [&](int64_t token) {
    routed = token < p.tokens && (p.mask == nullptr || p.mask[token] != 0);
    // one that is not stands for the first, so that the registers are loaded in every lane
    load_row<DT, EPL, RUNS>(p.logits + (routed ? token * p.ld : 0), slot, E, v);
  };
  if (p.tokens > 0) load(t);
  for (int64_t base = (int64_t)blockIdx.x * kFwdTokens; base < p.tokens;
       base += stride, t += stride) {
    // opaque: keeps what every expert's index gives from being held over the loop
    asm volatile("" : "+v"(slot));
    float ex[EPL];
    uint32_t key[EPL];
    close_absent<DT, EPL, RUNS>(v, routed, slot, E);
    Softmax sm = softmax(v, ex);
    const bool here = routed, nonfinite = !(sm.sum < INFINITY);
    bad |= nonfinite;
    const auto key_of = [&](float x, int j) {
      return (order(x) & ~255u) | (uint32_t)(255 - expert_of<DT, EPL, RUNS>(slot, j));
    };
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = key_of(v[j], j);
    if (__any(nonfinite)) {
      close_if_all_nan(v, ex, sm);
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = key_of(closed_if_nan(v[j]), j);
    }
    // the next tokens' logits, into the registers that are free now
    load(t + stride);
    wave_fence();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      acc[j] = fmaf(ex[j], sm.inv, acc[j]);
      mine[expert_of<DT, EPL, RUNS>(slot, j)] = ex[j];
    }
    wave_fence();
    live_tokens += sm.live ? 1 : 0;
    const int e = choose<DT, EPL, RUNS>(key, slot, E, k, [&](uint32_t (&whole)[EPL]) {
      float x[EPL];
#pragma unroll
      for (int j = 0; j < EPL; ++j) x[j] = -INFINITY;
      if (here) load_row<DT, EPL, RUNS>(p.logits + t * p.ld, slot, E, x);
      close_absent<DT, EPL, RUNS>(x, here, slot, E);
#pragma unroll
      for (int j = 0; j < EPL; ++j) whole[j] = order(closed_if_nan(x[j]));
    });
    float weight = e >= 0 ? mine[e] * sm.inv : 0.0f;
    if (p.normalize) {
      const float all = sum16(weight);
      weight = e >= 0 ? weight / all : 0.0f;
    }
    if (t < p.tokens && slot < k) {
      p.experts[t * k + slot] = e;
      p.weights[t * k + slot] = weight;
      if (e >= 0) atomicAdd(&hist[e], 1);
    }
  }
  __syncthreads();
  if (__any(bad) && lane == 0) dev_status_or(p.status, kDevNonFinite);
  // the wave's four tokens, then the waves
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    acc[j] += __shfl_xor(acc[j], 16, 64);
    acc[j] += __shfl_xor(acc[j], 32, 64);
    if (lane < kLanes) sums[w][expert_of<DT, EPL, RUNS>(slot, j)] = acc[j];
  }
  live_tokens += __shfl_xor(live_tokens, 16, 64);
  live_tokens += __shfl_xor(live_tokens, 32, 64);
  if (lane == 0) live_of[w] = live_tokens;
  __syncthreads();
  int live = 0;
#pragma unroll
  for (int i = 0; i < kFwdWaves; ++i) live += live_of[i];
  float sum = 0.0f;
  if (tid < E) {
#pragma unroll
    for (int i = 0; i < kFwdWaves; ++i) sum += sums[i][tid];
  }
  if (gridDim.x > 1) {
    if (tid < E) p.parts[(int64_t)blockIdx.x * E + tid] = v2i{__float_as_int(sum), hist[tid]};
    if (tid == 0) p.part_live[blockIdx.x] = live;
    return;
  }
  if (tid < kMaxExperts) {
    const double c = wave_sum(tid < E ? (double)hist[tid] * sum : 0.0);
    if (lane == 0) products[w] = c;
    if (tid < E) {
      p.counts[tid] = hist[tid];
      p.prob_sums[tid] = sum;
    }
  }
  __syncthreads();
  if (tid == 0) {
    *p.live = live;
    *p.loss = balance_loss(products[0] + products[1] + products[2] + products[3], E, k, live);
  }
}

// Adds up the workgroups' sums: 16 experts a workgroup, 16 threads an expert.  The last
// workgroup to end adds up the loss.
constexpr int kFinishThreads = 1024, kFinishParts = kFinishThreads / 16,
              kFinishWaves = kFinishThreads / 64;

__global__ __launch_bounds__(kFinishThreads) void router_finish_kernel(Fwd p, int parts) {
  __shared__ double sums[kFinishWaves][16];
  __shared__ int32_t counts[kFinishWaves][16];
  __shared__ bool last;
  __shared__ double waves[kFinishWaves];
  __shared__ int32_t lives[kFinishWaves];
  const int tid = threadIdx.x, e = tid & 15, i = tid >> 4;
  const int expert = (int)blockIdx.x * 16 + e;
  double s = 0.0;
  int32_t c = 0;
  if (expert < p.E) {
#pragma unroll 4
    for (int b = i; b < parts; b += kFinishParts) {
      const v2i v = p.parts[(int64_t)b * p.E + expert];
      const int bits = v[0];
      s += (double)__int_as_float(bits);
      c += v[1];
    }
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    s += __shfl_xor(s, d, 64);
    c += __shfl_xor(c, d, 64);
  }
  if ((tid & 63) < 16) {
    sums[tid >> 6][e] = s;
    counts[tid >> 6][e] = c;
  }
  __syncthreads();
  if (i == 0 && expert < p.E) {
#pragma unroll
    for (int j = 1; j < kFinishWaves; ++j) {
      s += sums[j][e];
      c += counts[j][e];
    }
    p.counts[expert] = c;
    p.prob_sums[expert] = (float)s;
    __hip_atomic_store(p.products + expert, (double)c * s, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  }
  // thread 0 releases what its own wave stored, and the products are read past the caches: no
  // other wave has to write a cache back (a fence of every thread: 5.6 instead of 4.7 us)
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(p.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  double all = tid < p.E ? __hip_atomic_load(p.products + tid, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT)
                         : 0.0;
  int live = 0;
  for (int b = tid; b < parts; b += kFinishThreads) live += p.part_live[b];
  all = wave_sum(all);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) live += __shfl_xor(live, d, 64);
  if ((tid & 63) == 0) {
    waves[tid >> 6] = all;
    lives[tid >> 6] = live;
  }
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int j = 1; j < kFinishWaves; ++j) {
      live += lives[j];
      all += waves[j];
    }
    *p.live = live;
    *p.loss = balance_loss(all, p.E, p.k, live);
  }
}
static_assert(kMaxExperts <= kFinishThreads && kFwdBlocks <= kFinishThreads, "a thread each");

// ---------------------------------------------------------------- backward

struct Bwd {
  const char* logits;
  int64_t ld, tokens;
  const uint8_t* mask;
  int E, k, normalize;
  const int32_t* experts;
  const float* d_weights;  // or null
  const int32_t* counts;
  const int32_t* live;
  const float* d_loss;     // or null
  char* out;
  int64_t ldo;
};

// What the slots add goes to the experts' lanes through LDS: a row of E floats a token,
// zeros but for the slots, which are cleared again after they were read.
template <int DT, int EPL, bool RUNS>
__global__ __launch_bounds__(kBwdThreads) void router_backward_kernel(Bwd p) {
  __shared__ __attribute__((aligned(16))) float slots[kBwdTokens][kLanes * EPL];
  __shared__ __attribute__((aligned(16))) float probs[kBwdTokens][kLanes * EPL];
  const int tid = threadIdx.x, lane = tid & 63;
  int slot = lane & (kLanes - 1);
  const int E = p.E, k = p.k;
  float* mine = slots[tid >> 4];
  float b[EPL];
  const int n = p.d_loss != nullptr ? *p.live : 0;
  const float f = n > 0 ? (float)((double)*p.d_loss * E / ((double)k * n * n)) : 0.0f;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = expert_of<DT, EPL, RUNS>(slot, j);
    mine[e] = 0.0f;
    b[j] = f != 0.0f && e < E ? f * (float)p.counts[e] : 0.0f;
  }
  const int64_t stride = (int64_t)gridDim.x * kBwdTokens;
  int64_t t = (int64_t)blockIdx.x * kBwdTokens + (tid >> 4);
  float v[EPL], next_dw = 0.0f;
  int next_e = -1;
  bool routed;
  const auto load = [&](int64_t token) {
    routed = token < p.tokens && (p.mask == nullptr || p.mask[token] != 0);
    next_e = -1;
    load_row<DT, EPL, RUNS>(p.logits + (routed ? token * p.ld : 0), slot, E, v);
    if (routed && slot < k && p.d_weights != nullptr) {
      next_e = p.experts[token * k + slot];
      next_dw = p.d_weights[token * k + slot];
    }
  };
  load(t);
  for (int64_t base = (int64_t)blockIdx.x * kBwdTokens; base < p.tokens;
       base += stride, t += stride) {
    // opaque: keeps what every expert's index gives from being held over the loop
    asm volatile("" : "+v"(slot));
    float prob[EPL];
    const int e = next_e >= 0 && next_e < E ? next_e : -1;
    const float dw = e >= 0 ? next_dw : 0.0f;
    close_absent<DT, EPL, RUNS>(v, routed, slot, E);
    Softmax sm = softmax(v, prob);
    if (__any(!(sm.sum < INFINITY))) close_if_all_nan(v, prob, sm);
    load(t + stride);
#pragma unroll
    for (int j = 0; j < EPL; ++j) prob[j] *= sm.inv;
    float add = dw;
    if (p.normalize) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) probs[tid >> 4][expert_of<DT, EPL, RUNS>(slot, j)] = prob[j];
      wave_fence();
      float weight = e >= 0 ? probs[tid >> 4][e] : 0.0f;
      const float all = sum16(weight);
      weight = e >= 0 ? weight / all : 0.0f;
      add = weight * (dw - sum16(e >= 0 ? weight * dw : 0.0f));
    }
    if (e >= 0) atomicAdd(&mine[e], add);
    wave_fence();
    float a[EPL], dot = 0.0f, given[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) given[j] = mine[expert_of<DT, EPL, RUNS>(slot, j)];
    wave_fence();
    if (e >= 0) mine[e] = 0.0f;
    wave_fence();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      a[j] = p.normalize ? b[j] : b[j] + given[j];
      dot += prob[j] * a[j];
    }
    dot = sum16(dot);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float d = prob[j] * (a[j] - dot) + (p.normalize ? given[j] : 0.0f);
      a[j] = sm.live ? d : 0.0f;
    }
    if (t < p.tokens) store_row<DT, EPL, RUNS>(p.out + t * p.ldo, slot, E, a);
  }
}

// f<DT, EPL, RUNS> for a type and a number of experts.
template <int DT, int EPL, typename F>
hipError_t by_runs(int E, F f) {
  const std::integral_constant<int, DT> dt;
  const std::integral_constant<int, EPL> epl;
  if constexpr (EPL > 1)
    if (E % kRun<DT, EPL, true> != 0) return f(dt, epl, std::false_type{});
  return f(dt, epl, std::true_type{});
}
template <int DT, typename F>
hipError_t by_experts(int E, F f) {
  if (E <= 16) return by_runs<DT, 1>(E, f);
  if (E <= 32) return by_runs<DT, 2>(E, f);
  if (E <= 64) return by_runs<DT, 4>(E, f);
  if (E <= 128) return by_runs<DT, 8>(E, f);
  return by_runs<DT, 16>(E, f);
}
template <typename F>
hipError_t by_type(int dtype, int E, F f) {
  if (dtype == 0) return by_experts<0>(E, f);
  if (dtype == 1) return by_experts<1>(E, f);
  return by_experts<2>(E, f);
}

int element_bytes(int dtype) { return dtype == 2 ? 4 : 2; }

}  // namespace

// The same for every number of tokens, and more for more experts.
size_t router_workspace_bytes(int64_t E) {
  return 64 + 4 * (size_t)kFwdBlocks + 8 * (size_t)E + 8 * (size_t)kFwdBlocks * (size_t)E;
}

hipError_t launch_router(int dtype, const void* logits, int64_t ld, int64_t tokens, int E, int k,
                         const uint8_t* mask, int normalize, int32_t* experts, float* weights,
                         int32_t* counts, float* prob_sums, int32_t* live, float* loss, void* ws,
                         uint32_t* status, hipStream_t stream) {
  Fwd p{};
  p.logits = static_cast<const char*>(logits);
  p.ld = ld * element_bytes(dtype);
  p.tokens = tokens;
  p.mask = mask;
  p.E = E; p.k = k; p.normalize = normalize;
  p.experts = experts; p.weights = weights; p.counts = counts; p.prob_sums = prob_sums;
  p.live = live; p.loss = loss; p.status = status;
  char* at = static_cast<char*>(ws);
  p.done = reinterpret_cast<uint32_t*>(at);
  at += 64;
  p.products = reinterpret_cast<double*>(at);
  at += 8 * (size_t)E;
  p.part_live = reinterpret_cast<int32_t*>(at);
  at += 4 * (size_t)kFwdBlocks;
  p.parts = reinterpret_cast<v2i*>(at);
  const int64_t want = (tokens + kFwdTokens - 1) / kFwdTokens;
  const int blocks = tokens <= kOneBlock ? 1 : (int)(want < kFwdBlocks ? want : kFwdBlocks);
  const hipError_t e = by_type(dtype, E, [&](auto dt, auto epl, auto runs) {
    constexpr int DT = decltype(dt)::value, EPL = decltype(epl)::value;
    hipLaunchKernelGGL((router_kernel<DT, EPL, decltype(runs)::value>), dim3(blocks),
                       dim3(kFwdThreads), 0, stream, p);
    return hipGetLastError();
  });
  if (e != hipSuccess || blocks == 1) return e;
  hipLaunchKernelGGL(router_finish_kernel, dim3((E + 15) / 16), dim3(kFinishThreads), 0, stream, p,
                     blocks);
  return hipGetLastError();
}

hipError_t launch_router_backward(int dtype, const void* logits, int64_t ld, int64_t tokens, int E,
                                  int k, const uint8_t* mask, int normalize, const int32_t* experts,
                                  const float* d_weights, const int32_t* counts,
                                  const int32_t* live, const float* d_loss, void* out, int64_t ldo,
                                  hipStream_t stream) {
  if (tokens == 0) return hipSuccess;
  Bwd p{};
  p.logits = static_cast<const char*>(logits);
  p.ld = ld * element_bytes(dtype);
  p.tokens = tokens;
  p.mask = mask;
  p.E = E; p.k = k; p.normalize = normalize;
  p.experts = experts; p.d_weights = d_weights; p.counts = counts; p.live = live;
  p.d_loss = d_loss;
  p.out = static_cast<char*>(out);
  p.ldo = ldo * element_bytes(dtype);
  const int64_t want = (tokens + kBwdTokens - 1) / kBwdTokens;
  const int64_t cap = 4 * (int64_t)device_cu_count();
  const unsigned blocks = (unsigned)(want < cap ? want : cap);
  return by_type(dtype, E, [&](auto dt, auto epl, auto runs) {
    constexpr int DT = decltype(dt)::value, EPL = decltype(epl)::value;
    hipLaunchKernelGGL((router_backward_kernel<DT, EPL, decltype(runs)::value>), dim3(blocks),
                       dim3(kBwdThreads), 0, stream, p);
    return hipGetLastError();
  });
}

}  // namespace bsg
