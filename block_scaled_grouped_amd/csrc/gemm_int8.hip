// Products of 8-bit integers with a scale for each token and each channel:
//
//   Y[r, j] = (float32(sum_i A[r, i] B_g[j, i]) * a_scales[r]) * b_scales[g, j]
//
// on the tiles of the 16-bit products (INT8 there).  The sums are exact in 32 bits for
// contractions under 2^17, so splitting one changes nothing.
#include "gemm_large.h"
#include "gemm_small.h"

namespace bsg {

using namespace g16;

namespace g16 {

hipError_t launch_large_int8(int f16, const Args& p, hipStream_t stream) {
  return f16 ? large::launch<kInt8, true>(p, stream) : large::launch<kInt8, false>(p, stream);
}

namespace {

template <bool F16>
hipError_t launch_bm(int bm, const Args& p, hipStream_t stream) {
  if (bm <= 32) return small::launch<kInt8, F16, 32>(p, stream);
  if (bm <= 64) return small::launch<kInt8, F16, 64>(p, stream);
  return small::launch<kInt8, F16, 128>(p, stream);
}

}  // namespace

hipError_t launch_small_int8(int f16, int bm, const Args& p, hipStream_t stream) {
  return f16 ? launch_bm<true>(bm, p, stream) : launch_bm<false>(bm, p, stream);
}

}  // namespace g16

namespace {

// Whether the form of few rows runs.  It reads a group's weights once for 16 rows, the 32-row
// tiles once for 32, at a lower rate and with a second step for split contractions.  us, few
// rows and 32-row tiles, n x k 4096 x 4096: 16 rows of one group 9.7 and 14.2, 32 of eight 29.1
// and 29.9, 64 of eight 30.5 and 30.3, 128 of eight 36 and 32; 2048 x 7168: 64 of 64 107 and
// 118, 256 of 64 155 and 155.  Group sizes are on the device, and all rows may be one group's:
// the second bound keeps that case's price down.
bool few_rows(int64_t G, int64_t rows_cap) {
  return rows_cap <= 16 || (rows_cap <= 4 * G && rows_cap <= 256);
}

}  // namespace

int gemm_int8_tile_rows(int64_t G, int64_t rows_cap, int64_t n, int64_t k, bool split) {
  return few_rows(G, rows_cap) ? 16 : form_rows(kInt8, G, rows_cap, n, k / 2, split);
}

hipError_t launch_gemm_int8(int G, const int8_t* a, int64_t lda, const float* a_scales,
                            const int8_t* b, int64_t ldb, int64_t stride_b, const float* b_scales,
                            const int64_t* offsets, int64_t rows_cap, int64_t n, int64_t k,
                            void* out, int64_t ldo, int f16, int out_f32, void* ws,
                            uint32_t* status, hipStream_t stream) {
  if (few_rows(G, rows_cap))
    return launch_gemm_int8_few(0, 0, G, a, lda, a_scales, b, ldb, stride_b, b_scales, offsets,
                                rows_cap, n, k, out, ldo, f16, out_f32, status, stream);
  Args p{};
  p.a = reinterpret_cast<const uint16_t*>(a);
  p.b = reinterpret_cast<const uint16_t*>(b);
  p.offsets = offsets;
  p.out = static_cast<char*>(out);
  p.lda = lda / 2; p.ldb = ldb / 2; p.stride_b = stride_b / 2; p.ldo = ldo;
  p.rows_cap = rows_cap; p.n = n; p.k = k / 2;
  p.status = status;
  p.ws = static_cast<char*>(ws);
  p.G = G; p.out_f32 = out_f32;
  p.a_scales = a_scales;
  p.b_scales = b_scales;
  const int bm = form_rows(kInt8, G, rows_cap, n, p.k, ws != nullptr);
  return bm == 256 ? launch_large_int8(f16, p, stream) : launch_small_int8(f16, bm, p, stream);
}

namespace {
size_t align256(int64_t n) { return (size_t)(n + 255) / 256 * 256; }
}  // namespace

size_t gemm_int8_dynamic_workspace_bytes(int64_t rows_cap, int64_t k) {
  return gemm_16bit_workspace_bytes() + align256(4 * rows_cap) + align256(rows_cap * k);
}

hipError_t launch_gemm_int8_dynamic(int in_f16, int G, const void* x, int64_t ldx, const int8_t* b,
                                    int64_t ldb, int64_t stride_b, const float* b_scales,
                                    const int64_t* offsets, int64_t rows_cap, int64_t n, int64_t k,
                                    void* out, int64_t ldo, int f16, int out_f32, void* ws,
                                    uint32_t* status, hipStream_t stream) {
  // a workgroup quantizes up to kFewTokenBytes of tokens faster than a launch of their own
  // takes (4096 columns: 1 row 9.6 and 12.5 us, 4 rows 19 and 15)
  if (rows_cap <= 8 && rows_cap * k <= kFewTokenBytes)
    return launch_gemm_int8_few(1, in_f16, G, x, ldx, nullptr, b, ldb, stride_b, b_scales, offsets,
                                rows_cap, n, k, out, ldo, f16, out_f32, status, stream);
  char* at = static_cast<char*>(ws) + gemm_16bit_workspace_bytes();
  float* scales = reinterpret_cast<float*>(at);
  int8_t* data = reinterpret_cast<int8_t*>(at + align256(4 * rows_cap));
  const hipError_t e = launch_quantize_int8(in_f16, x, ldx, rows_cap, k, G, offsets, data, scales,
                                            status, stream);
  if (e != hipSuccess) return e;
  return launch_gemm_int8(G, data, k, scales, b, ldb, stride_b, b_scales, offsets, rows_cap, n, k,
                          out, ldo, f16, out_f32, ws, status, stream);
}

}  // namespace bsg
