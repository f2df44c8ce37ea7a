// C-ABI entry points of libbsg (declared in include/bsg.h): host-side argument
// validation, then the kernel launchers.  No allocation, no synchronization, no
// device reads from the host.
#include "../../include/bsg.h"

#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "bsg_internal.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return BSG_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int hip_result(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(BSG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

// Largest byte span a single GEMM / quantize tile addresses with 32-bit offsets.
constexpr int64_t kMaxTileBytes = (int64_t)1 << 31;

}  // namespace

extern "C" {

const char* bsg_last_error(void) { return g_err; }

int bsg_version(void) { return (0 << 16) | 1; }

int group_offsets_i32_to_i64(const int32_t* sizes, int64_t G, int64_t multiplier, int64_t pad_to,
                             int64_t* sizes_i64, int64_t* offsets, int64_t capacity,
                             uint32_t* dev_status, void* stream) {
  if (sizes == nullptr || offsets == nullptr)
    return fail(BSG_ERR_NULL, "group_offsets_i32_to_i64: sizes and offsets must be non-NULL");
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "group_offsets_i32_to_i64: G=%lld outside [1, %d]", (long long)G,
                BSG_MAX_GROUPS);
  if (multiplier < 1 || pad_to < 1)
    return fail(BSG_ERR_SHAPE, "group_offsets_i32_to_i64: multiplier=%lld and pad_to=%lld must be >= 1",
                (long long)multiplier, (long long)pad_to);
  if (((int64_t)1 << 31) * pad_to > ((int64_t)1 << 62) / multiplier)
    return fail(BSG_ERR_SHAPE, "group_offsets_i32_to_i64: multiplier * pad_to too large");
  return hip_result(bsg::launch_group_offsets(sizes, (int)G, multiplier, pad_to, sizes_i64, offsets,
                                              capacity, dev_status, (hipStream_t)stream),
                    "group_offsets_i32_to_i64");
}

int grouped_quantize_mxfp8(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                           const int64_t* offsets, uint8_t* row_data, uint8_t* row_scales,
                           const int64_t* padded_offsets, int64_t col_rows_cap, uint8_t* col_data,
                           uint8_t* col_scales, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_mxfp8";
  if (x == nullptr || offsets == nullptr) return fail(BSG_ERR_NULL, "%s: x and offsets must be non-NULL", fn);
  const bool row = row_data != nullptr || row_scales != nullptr;
  const bool col = padded_offsets != nullptr || col_data != nullptr || col_scales != nullptr;
  if (row && (row_data == nullptr || row_scales == nullptr))
    return fail(BSG_ERR_NULL, "%s: row_data and row_scales go together", fn);
  if (col && (padded_offsets == nullptr || col_data == nullptr || col_scales == nullptr))
    return fail(BSG_ERR_NULL, "%s: padded_offsets, col_data and col_scales go together", fn);
  if (!row && !col) return fail(BSG_ERR_NULL, "%s: no output requested", fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and cols a positive multiple of 32 (got %lld, %lld)",
                fn, (long long)rows_cap, (long long)cols);
  if (col && (col_rows_cap < 0 || col_rows_cap * cols >= ((int64_t)1 << 40)))
    return fail(BSG_ERR_SHAPE, "%s: col_rows_cap=%lld out of range", fn, (long long)col_rows_cap);
  if (!aligned16(x) || (row && !aligned16(row_data)) || (col && !aligned16(col_data)))
    return fail(BSG_ERR_ALIGN, "%s: x, row_data and col_data must be 16-byte aligned", fn);
  if (row && !aligned4(row_scales))
    return fail(BSG_ERR_ALIGN, "%s: row_scales must be 4-byte aligned", fn);
  hipStream_t s = (hipStream_t)stream;
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  if (col) {
    // one pass over x for both directions when both are requested
    return hip_result(bsg::launch_quantize_mxfp8_colwise(xb, rows_cap, cols, (int)G, offsets,
                                                         padded_offsets, col_rows_cap, col_data,
                                                         col_scales, row ? row_data : nullptr,
                                                         row ? row_scales : nullptr, dev_status, s),
                      fn);
  }
  return hip_result(bsg::launch_quantize_mxfp8_rowwise(xb, rows_cap, cols, (int)G, offsets, row_data,
                                                       row_scales, dev_status, s),
                    fn);
}

int grouped_quantize_mxfp8_colwise_e5m2(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                                        const int64_t* offsets, const int64_t* padded_offsets,
                                        int64_t col_rows_cap, uint8_t* col_data,
                                        uint8_t* col_scales, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_mxfp8_colwise_e5m2";
  if (x == nullptr || offsets == nullptr || padded_offsets == nullptr || col_data == nullptr ||
      col_scales == nullptr)
    return fail(BSG_ERR_NULL, "%s: x, offsets, padded_offsets, col_data and col_scales must be non-NULL",
                fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and cols a positive multiple of 32 (got %lld, %lld)",
                fn, (long long)rows_cap, (long long)cols);
  if (col_rows_cap < 0 || col_rows_cap * cols >= ((int64_t)1 << 40))
    return fail(BSG_ERR_SHAPE, "%s: col_rows_cap=%lld out of range", fn, (long long)col_rows_cap);
  if (!aligned16(x) || !aligned16(col_data))
    return fail(BSG_ERR_ALIGN, "%s: x and col_data must be 16-byte aligned", fn);
  return hip_result(bsg::launch_quantize_mxfp8_colwise(static_cast<const uint16_t*>(x), rows_cap,
                                                       cols, (int)G, offsets, padded_offsets,
                                                       col_rows_cap, col_data, col_scales, nullptr,
                                                       nullptr, dev_status, (hipStream_t)stream,
                                                       true),
                    fn);
}

int grouped_quantize_mxfp8_rowwise_e5m2(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                                        const int64_t* offsets, uint8_t* row_data,
                                        uint8_t* row_scales, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_mxfp8_rowwise_e5m2";
  if (x == nullptr || offsets == nullptr || row_data == nullptr || row_scales == nullptr)
    return fail(BSG_ERR_NULL, "%s: x, offsets, row_data and row_scales must be non-NULL", fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and cols a positive multiple of 32 (got %lld, %lld)",
                fn, (long long)rows_cap, (long long)cols);
  if (!aligned16(x) || !aligned16(row_data) || !aligned4(row_scales))
    return fail(BSG_ERR_ALIGN, "%s: x and row_data must be 16-byte aligned, row_scales 4-byte", fn);
  return hip_result(bsg::launch_quantize_mxfp8_rowwise(static_cast<const uint16_t*>(x), rows_cap,
                                                       cols, (int)G, offsets, row_data, row_scales,
                                                       dev_status, (hipStream_t)stream, true),
                    fn);
}

int grouped_quantize_nvfp4_rowscaled(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                                     const int64_t* offsets, uint8_t* data, uint8_t* block_scales,
                                     float* outer, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_nvfp4_rowscaled";
  if (x == nullptr || offsets == nullptr || data == nullptr || block_scales == nullptr || outer == nullptr)
    return fail(BSG_ERR_NULL, "%s: x, offsets, data, block_scales and outer must be non-NULL", fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and cols a positive multiple of 32", fn);
  if (rows_cap > 0x7fffffffLL) return fail(BSG_ERR_SHAPE, "%s: rows_cap too large", fn);
  if (!aligned16(x) || !aligned16(data) || !aligned4(outer))
    return fail(BSG_ERR_ALIGN, "%s: x and data must be 16-byte aligned, outer 4-byte", fn);
  return hip_result(bsg::launch_quantize_nvfp4_rowscaled(static_cast<const uint16_t*>(x), rows_cap,
                                                         cols, (int)G, offsets, data, block_scales,
                                                         outer, dev_status, (hipStream_t)stream),
                    fn);
}

int grouped_quantize_nvfp4_pertensor(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                                     const int64_t* offsets, uint8_t* data, uint8_t* block_scales,
                                     float* amax, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_nvfp4_pertensor";
  if (x == nullptr || offsets == nullptr || data == nullptr || block_scales == nullptr || amax == nullptr)
    return fail(BSG_ERR_NULL, "%s: x, offsets, data, block_scales and amax must be non-NULL", fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and cols a positive multiple of 32", fn);
  if (rows_cap > 0x7fffffffLL) return fail(BSG_ERR_SHAPE, "%s: rows_cap too large", fn);
  if (!aligned16(x) || !aligned16(data) || !aligned4(amax))
    return fail(BSG_ERR_ALIGN, "%s: x and data must be 16-byte aligned, amax 4-byte", fn);
  return hip_result(bsg::launch_quantize_nvfp4_pertensor(static_cast<const uint16_t*>(x), rows_cap,
                                                         cols, (int)G, offsets, data, block_scales,
                                                         amax, dev_status, (hipStream_t)stream),
                    fn);
}

static int pertensor_args(const char* fn, const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                          const int64_t* offsets, const uint8_t* data, const uint8_t* block_scales,
                          const float* amax) {
  if (x == nullptr || offsets == nullptr || data == nullptr || block_scales == nullptr || amax == nullptr)
    return fail(BSG_ERR_NULL, "%s: x, offsets, data, block_scales and amax must be non-NULL", fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and cols a positive multiple of 32", fn);
  if (rows_cap > 0x7fffffffLL) return fail(BSG_ERR_SHAPE, "%s: rows_cap too large", fn);
  if (!aligned16(x) || !aligned16(data) || !aligned4(amax))
    return fail(BSG_ERR_ALIGN, "%s: x and data must be 16-byte aligned, amax 4-byte", fn);
  return BSG_OK;
}

int grouped_quantize_nvfp4_pertensor_rht(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                                         const int64_t* offsets, uint32_t rht_sign_mask,
                                         uint8_t* data, uint8_t* block_scales, float* amax,
                                         uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_nvfp4_pertensor_rht";
  const int rc = pertensor_args(fn, x, rows_cap, cols, G, offsets, data, block_scales, amax);
  if (rc != BSG_OK) return rc;
  if (rht_sign_mask > 0xffffu)
    return fail(BSG_ERR_SHAPE, "%s: rht_sign_mask has bits above the 16 signs", fn);
  return hip_result(bsg::launch_quantize_nvfp4_pertensor_rht(static_cast<const uint16_t*>(x),
                                                             rows_cap, cols, (int)G, offsets,
                                                             rht_sign_mask, data, block_scales,
                                                             amax, dev_status, (hipStream_t)stream),
                    fn);
}

int grouped_quantize_nvfp4_pertensor_2d(const void* x, int64_t rows_cap, int64_t cols, int64_t G,
                                        const int64_t* offsets, uint8_t* data,
                                        uint8_t* block_scales, float* amax, uint32_t* dev_status,
                                        void* stream) {
  const char* fn = "grouped_quantize_nvfp4_pertensor_2d";
  const int rc = pertensor_args(fn, x, rows_cap, cols, G, offsets, data, block_scales, amax);
  if (rc != BSG_OK) return rc;
  return hip_result(bsg::launch_quantize_nvfp4_pertensor_2d(static_cast<const uint16_t*>(x),
                                                            rows_cap, cols, (int)G, offsets, data,
                                                            block_scales, amax, dev_status,
                                                            (hipStream_t)stream),
                    fn);
}

int grouped_quantize_nvfp4_rowscaled_colwise(const void* x, int64_t rows_cap, int64_t cols,
                                             int64_t G, const int64_t* offsets,
                                             const int64_t* padded_offsets, int64_t col_rows_cap,
                                             uint8_t* data, uint8_t* block_scales, float* outer,
                                             uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_quantize_nvfp4_rowscaled_colwise";
  if (x == nullptr || offsets == nullptr || padded_offsets == nullptr || data == nullptr ||
      block_scales == nullptr || outer == nullptr)
    return fail(BSG_ERR_NULL,
                "%s: x, offsets, padded_offsets, data, block_scales and outer must be non-NULL", fn);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || col_rows_cap < 0 || cols <= 0 || cols % 32 != 0)
    return fail(BSG_ERR_SHAPE,
                "%s: need rows_cap >= 0, col_rows_cap >= 0 and cols a positive multiple of 32", fn);
  if (rows_cap > 0x7fffffffLL || col_rows_cap > 0x7fffffffLL)
    return fail(BSG_ERR_SHAPE, "%s: rows_cap or col_rows_cap too large", fn);
  if (!aligned16(x) || !aligned16(data) || !aligned4(outer))
    return fail(BSG_ERR_ALIGN, "%s: x and data must be 16-byte aligned, outer 4-byte", fn);
  return hip_result(bsg::launch_quantize_nvfp4_rowscaled_colwise(
                        static_cast<const uint16_t*>(x), rows_cap, cols, (int)G, offsets,
                        padded_offsets, col_rows_cap, data, block_scales, outer, dev_status,
                        (hipStream_t)stream),
                    fn);
}

static int gemm_mxfp8_impl(const char* fn, int mode, int64_t G, const uint8_t* a,
                           const uint8_t* a_scales, const uint8_t* b, const uint8_t* b_scales,
                           const int64_t* offsets, int64_t rows_cap, int64_t n, int64_t k,
                           void* out, int out_dtype, const float* alpha, const float* beta,
                           const float* bias, uint32_t* dev_status, void* stream,
                           void* ws = nullptr) {
  if (a == nullptr || a_scales == nullptr || b == nullptr || b_scales == nullptr || offsets == nullptr ||
      out == nullptr)
    return fail(BSG_ERR_NULL, "%s: operands, scales, offsets and out must be non-NULL", fn);
  if (mode != BSG_FPROP_TN && mode != BSG_WGRAD_NT && mode != BSG_DGRAD_NN &&
      mode != BSG_WGRAD_NT_E5M2)
    return fail(BSG_ERR_UNSUPPORTED, "%s: unknown mode %d", fn, mode);
  if (out_dtype != BSG_OUT_BF16 && out_dtype != BSG_OUT_F32)
    return fail(BSG_ERR_UNSUPPORTED, "%s: unknown out_dtype %d", fn, out_dtype);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || n < 1 || k < 1)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0, n >= 1, k >= 1", fn);
  const int64_t esz = out_dtype == BSG_OUT_F32 ? 4 : 2;
  const bool wgrad = mode == BSG_WGRAD_NT || mode == BSG_WGRAD_NT_E5M2;
  if (!wgrad) {
    if (k % 32 != 0)
      return fail(BSG_ERR_SHAPE, "%s: FPROP / DGRAD need k %% 32 == 0 (got %lld)", fn, (long long)k);
    const int64_t nq = (k + 127) / 128;  // scale words per row; DGRAD's B rows hold 128 nq bytes
    if (256 * 128 * nq >= kMaxTileBytes || 256 * n * esz >= kMaxTileBytes || n > 0x7fffffffLL)
      return fail(BSG_ERR_SHAPE, "%s: n or k too large for one tile's 32-bit offsets", fn);
    if (nq * 4 * rows_cap >= kMaxTileBytes || nq * 4 * G * n >= kMaxTileBytes)
      return fail(BSG_ERR_SHAPE, "%s: scale arrays too large for 32-bit offsets", fn);
  } else {
    if (n % 32 != 0 || k % 32 != 0)
      return fail(BSG_ERR_SHAPE, "%s: WGRAD needs n and k multiples of 32", fn);
    if (256 * rows_cap >= kMaxTileBytes || 256 * k * esz >= kMaxTileBytes ||
        (rows_cap / 128) * 4 * (n > k ? n : k) >= kMaxTileBytes)
      return fail(BSG_ERR_SHAPE, "%s: token capacity or k too large for 32-bit tile offsets", fn);
  }
  if (!aligned16(a) || !aligned16(b) || !aligned4(a_scales) || !aligned4(b_scales) || !aligned4(out))
    return fail(BSG_ERR_ALIGN, "%s: a and b must be 16-byte aligned; scales and out 4-byte", fn);
  if (!aligned4(alpha) || !aligned4(beta) || !aligned16(bias))
    return fail(BSG_ERR_ALIGN, "%s: alpha and beta must be 4-byte aligned, bias 16-byte", fn);
  if (bias != nullptr && ((wgrad ? k : n) % 4 != 0))
    return fail(BSG_ERR_SHAPE, "%s: a bias needs a multiple of 4 output columns", fn);
  return hip_result(bsg::launch_gemm_mxfp8(mode, (int)G, a, a_scales, b, b_scales, offsets, rows_cap,
                                           n, k, out, out_dtype == BSG_OUT_F32, dev_status,
                                           (hipStream_t)stream, alpha, beta, bias, ws),
                    fn);
}

int grouped_gemm_mxfp8(int mode, int64_t G, const uint8_t* a, const uint8_t* a_scales,
                       const uint8_t* b, const uint8_t* b_scales, const int64_t* offsets,
                       int64_t rows_cap, int64_t n, int64_t k, void* out, int out_dtype,
                       uint32_t* dev_status, void* stream) {
  return gemm_mxfp8_impl("grouped_gemm_mxfp8", mode, G, a, a_scales, b, b_scales, offsets,
                         rows_cap, n, k, out, out_dtype, nullptr, nullptr, nullptr, dev_status,
                         stream);
}

size_t grouped_gemm_mxfp8_workspace_size(void) { return bsg::gemm_mxfp8_workspace_bytes(); }

int grouped_gemm_mxfp8_ws(int mode, int64_t G, const uint8_t* a, const uint8_t* a_scales,
                          const uint8_t* b, const uint8_t* b_scales, const int64_t* offsets,
                          int64_t rows_cap, int64_t n, int64_t k, void* out, int out_dtype,
                          void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                          void* stream) {
  const char* fn = "grouped_gemm_mxfp8_ws";
  if (workspace == nullptr) return fail(BSG_ERR_NULL, "%s: workspace is NULL", fn);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(BSG_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  const size_t need = bsg::gemm_mxfp8_workspace_bytes();
  if (workspace_bytes < need)
    return fail(BSG_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes,
                need);
  return gemm_mxfp8_impl(fn, mode, G, a, a_scales, b, b_scales, offsets, rows_cap, n, k, out,
                         out_dtype, nullptr, nullptr, nullptr, dev_status, stream, workspace);
}

int grouped_gemm_mxfp8_ex(int mode, int64_t G, const uint8_t* a, const uint8_t* a_scales,
                          const uint8_t* b, const uint8_t* b_scales, const int64_t* offsets,
                          int64_t rows_cap, int64_t n, int64_t k, void* out, int out_dtype,
                          const float* alpha, const float* beta, const float* bias,
                          uint32_t* dev_status, void* stream) {
  return gemm_mxfp8_impl("grouped_gemm_mxfp8_ex", mode, G, a, a_scales, b, b_scales, offsets,
                         rows_cap, n, k, out, out_dtype, alpha, beta, bias, dev_status, stream);
}

static int gemm_nvfp4_impl(const char* fn, bool per_tensor, int64_t G, const uint8_t* a,
                           const uint8_t* a_scales, const float* a_outer, const int64_t* offsets,
                           int64_t rows_cap, int64_t k, const uint8_t* b, const uint8_t* b_scales,
                           const float* b_outer, const int64_t* n_per_group, void* out,
                           int64_t ld_out, int out_dtype, float* scratch, uint32_t* dev_status,
                           void* stream, bool noalloc = false, bool accumulate = false,
                           void* ws = nullptr) {
  if (a == nullptr || a_scales == nullptr || a_outer == nullptr || offsets == nullptr || b == nullptr ||
      b_scales == nullptr || b_outer == nullptr || n_per_group == nullptr || out == nullptr)
    return fail(BSG_ERR_NULL, "%s: operands, scales, offsets, n_per_group and out must be non-NULL", fn);
  if (out_dtype != BSG_OUT_BF16 && out_dtype != BSG_OUT_F32)
    return fail(BSG_ERR_UNSUPPORTED, "%s: unknown out_dtype %d", fn, out_dtype);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || k < 32 || k % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need rows_cap >= 0 and k a positive multiple of 32 (got %lld)", fn,
                (long long)k);
  bsg::NvGroupTable tab;
  memset(&tab, 0, sizeof tab);
  int64_t max_n = 0, brow = 0;
  for (int64_t g = 0; g < G; ++g) {
    const int64_t ng = n_per_group[g];
    if (ng < 0 || ng > 0x7fffffffLL) return fail(BSG_ERR_SHAPE, "%s: n_per_group[%lld] out of range", fn, (long long)g);
    tab.n[g] = (int32_t)ng;
    tab.brow[g] = (int32_t)brow;
    brow += ng;
    if (brow > 0x7fffffffLL) return fail(BSG_ERR_SHAPE, "%s: sum of n_per_group too large", fn);
    if (ng > max_n) max_n = ng;
  }
  tab.brow[G] = (int32_t)brow;
  if (ld_out < max_n || ld_out < 1)
    return fail(BSG_ERR_SHAPE, "%s: ld_out=%lld below the widest group (%lld)", fn, (long long)ld_out,
                (long long)max_n);
  if (noalloc && rows_cap * ld_out > (int64_t)(bsg::kNoAllocScratchBytes / sizeof(float)))
    return fail(BSG_ERR_SHAPE,
                "%s: rows_cap * ld_out * 4 = %lld bytes exceeds the library's %lld-byte static "
                "scratch; use grouped_gemm_nvfp4_rowscaled with a caller scratch",
                fn, (long long)(rows_cap * ld_out * 4), (long long)bsg::kNoAllocScratchBytes);
  const int64_t esz = (out_dtype == BSG_OUT_F32 || scratch != nullptr || noalloc) ? 4 : 2;
  if (256 * (k / 2) >= kMaxTileBytes || 256 * ld_out * esz >= kMaxTileBytes)
    return fail(BSG_ERR_SHAPE, "%s: k or ld_out too large for 32-bit tile offsets", fn);
  if (!aligned16(a) || !aligned16(b) || !aligned4(a_scales) || !aligned4(b_scales) || !aligned4(out) ||
      (scratch != nullptr && !aligned4(scratch)))
    return fail(BSG_ERR_ALIGN, "%s: a and b must be 16-byte aligned; scales, out and scratch 4-byte", fn);
  if (noalloc)
    return hip_result(bsg::launch_gemm_nvfp4_noalloc((int)G, a, a_scales, a_outer, offsets,
                                                     rows_cap, k, b, b_scales, b_outer, tab,
                                                     (int)max_n, out, ld_out,
                                                     out_dtype == BSG_OUT_F32, dev_status,
                                                     (hipStream_t)stream),
                      fn);
  return hip_result(bsg::launch_gemm_nvfp4((int)G, a, a_scales, a_outer, offsets, rows_cap, k, b,
                                           b_scales, b_outer, tab, (int)max_n, out, ld_out,
                                           out_dtype == BSG_OUT_F32, scratch, dev_status,
                                           (hipStream_t)stream, per_tensor, accumulate, ws),
                    fn);
}

// Checks a split workspace argument; 0 when usable.
static int check_nvfp4_workspace(const char* fn, void* workspace, size_t workspace_bytes) {
  if (workspace == nullptr) return fail(BSG_ERR_NULL, "%s: workspace is NULL", fn);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(BSG_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  const size_t need = bsg::gemm_nvfp4_workspace_bytes();
  if (workspace_bytes < need)
    return fail(BSG_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes,
                need);
  return BSG_OK;
}

size_t grouped_gemm_nvfp4_workspace_size(void) { return bsg::gemm_nvfp4_workspace_bytes(); }

int grouped_gemm_nvfp4_rowscaled_ws(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                    const float* a_outer, const int64_t* offsets, int64_t rows_cap,
                                    int64_t k, const uint8_t* b, const uint8_t* b_scales,
                                    const float* b_outer, const int64_t* n_per_group, void* out,
                                    int64_t ld_out, int out_dtype, int accumulate, void* workspace,
                                    size_t workspace_bytes, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_gemm_nvfp4_rowscaled_ws";
  if (accumulate != 0 && accumulate != 1)
    return fail(BSG_ERR_UNSUPPORTED, "%s: accumulate must be 0 or 1", fn);
  const int wc = check_nvfp4_workspace(fn, workspace, workspace_bytes);
  if (wc != BSG_OK) return wc;
  return gemm_nvfp4_impl(fn, false, G, a, a_scales, a_outer, offsets, rows_cap, k, b, b_scales,
                         b_outer, n_per_group, out, ld_out, out_dtype, nullptr, dev_status, stream,
                         false, accumulate == 1, workspace);
}

int grouped_gemm_nvfp4_pertensor_ws(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                    const float* a_amax, const int64_t* offsets, int64_t rows_cap,
                                    int64_t k, const uint8_t* b, const uint8_t* b_scales,
                                    const float* b_amax, const int64_t* n_per_group, void* out,
                                    int64_t ld_out, int out_dtype, void* workspace,
                                    size_t workspace_bytes, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_gemm_nvfp4_pertensor_ws";
  const int wc = check_nvfp4_workspace(fn, workspace, workspace_bytes);
  if (wc != BSG_OK) return wc;
  return gemm_nvfp4_impl(fn, true, G, a, a_scales, a_amax, offsets, rows_cap, k, b, b_scales,
                         b_amax, n_per_group, out, ld_out, out_dtype, nullptr, dev_status, stream,
                         false, false, workspace);
}

int grouped_gemm_nvfp4_rowscaled(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                 const float* a_outer, const int64_t* offsets, int64_t rows_cap,
                                 int64_t k, const uint8_t* b, const uint8_t* b_scales,
                                 const float* b_outer, const int64_t* n_per_group, void* out,
                                 int64_t ld_out, int out_dtype, float* scratch,
                                 uint32_t* dev_status, void* stream) {
  return gemm_nvfp4_impl("grouped_gemm_nvfp4_rowscaled", false, G, a, a_scales, a_outer, offsets,
                         rows_cap, k, b, b_scales, b_outer, n_per_group, out, ld_out, out_dtype,
                         scratch, dev_status, stream);
}

int grouped_gemm_nvfp4_rowscaled_ex(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                    const float* a_outer, const int64_t* offsets, int64_t rows_cap,
                                    int64_t k, const uint8_t* b, const uint8_t* b_scales,
                                    const float* b_outer, const int64_t* n_per_group, void* out,
                                    int64_t ld_out, int out_dtype, float* scratch, int accumulate,
                                    uint32_t* dev_status, void* stream) {
  if (accumulate != 0 && accumulate != 1)
    return fail(BSG_ERR_UNSUPPORTED, "grouped_gemm_nvfp4_rowscaled_ex: accumulate must be 0 or 1");
  return gemm_nvfp4_impl("grouped_gemm_nvfp4_rowscaled_ex", false, G, a, a_scales, a_outer, offsets,
                         rows_cap, k, b, b_scales, b_outer, n_per_group, out, ld_out, out_dtype,
                         scratch, dev_status, stream, false, accumulate == 1);
}

int grouped_gemm_nvfp4_rowscaled_noalloc(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                         const float* a_outer, const int64_t* offsets,
                                         int64_t rows_cap, int64_t k, const uint8_t* b,
                                         const uint8_t* b_scales, const float* b_outer,
                                         const int64_t* n_per_group, void* out, int64_t ld_out,
                                         int out_dtype, uint32_t* dev_status, void* stream) {
  return gemm_nvfp4_impl("grouped_gemm_nvfp4_rowscaled_noalloc", false, G, a, a_scales, a_outer,
                         offsets, rows_cap, k, b, b_scales, b_outer, n_per_group, out, ld_out,
                         out_dtype, nullptr, dev_status, stream, true);
}

int grouped_gemm_nvfp4_pertensor(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                 const float* a_amax, const int64_t* offsets, int64_t rows_cap,
                                 int64_t k, const uint8_t* b, const uint8_t* b_scales,
                                 const float* b_amax, const int64_t* n_per_group, void* out,
                                 int64_t ld_out, int out_dtype, uint32_t* dev_status, void* stream) {
  return gemm_nvfp4_impl("grouped_gemm_nvfp4_pertensor", true, G, a, a_scales, a_amax, offsets,
                         rows_cap, k, b, b_scales, b_amax, n_per_group, out, ld_out, out_dtype,
                         nullptr, dev_status, stream);
}

static int nv_wgrad_impl(const char* fn, int64_t G, const uint8_t* a, const uint8_t* a_scales,
                         const float* a_outer, const uint8_t* b, const uint8_t* b_scales,
                         const float* b_outer, const int64_t* padded_offsets, int64_t col_rows_cap,
                         int64_t n, int64_t k, void* out, int out_dtype, bool accumulate,
                         uint32_t* dev_status, void* stream) {
  if (a == nullptr || a_scales == nullptr || a_outer == nullptr || b == nullptr ||
      b_scales == nullptr || b_outer == nullptr || padded_offsets == nullptr || out == nullptr)
    return fail(BSG_ERR_NULL, "%s: operands, scales, padded_offsets and out must be non-NULL", fn);
  if (out_dtype != BSG_OUT_BF16 && out_dtype != BSG_OUT_F32)
    return fail(BSG_ERR_UNSUPPORTED, "%s: unknown out_dtype %d", fn, out_dtype);
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (col_rows_cap < 0 || n < 32 || k < 32 || n % 32 != 0 || k % 32 != 0)
    return fail(BSG_ERR_SHAPE, "%s: need col_rows_cap >= 0 and n, k positive multiples of 32", fn);
  const int64_t esz = out_dtype == BSG_OUT_F32 ? 4 : 2;
  if (256 * (col_rows_cap / 2) >= kMaxTileBytes || 256 * k * esz >= kMaxTileBytes ||
      n > 0x7fffffffLL || k > 0x7fffffffLL)
    return fail(BSG_ERR_SHAPE, "%s: col_rows_cap, n or k too large for 32-bit tile offsets", fn);
  if (!aligned16(a) || !aligned16(b) || !aligned4(a_scales) || !aligned4(b_scales) ||
      !aligned4(a_outer) || !aligned4(b_outer) || !aligned4(out))
    return fail(BSG_ERR_ALIGN, "%s: a and b must be 16-byte aligned; scales, outer and out 4-byte",
                fn);
  return hip_result(bsg::launch_gemm_nvfp4_wgrad((int)G, a, a_scales, a_outer, b, b_scales,
                                                 b_outer, padded_offsets, col_rows_cap, n, k, out,
                                                 out_dtype == BSG_OUT_F32, dev_status,
                                                 (hipStream_t)stream, accumulate),
                    fn);
}

int grouped_gemm_nvfp4_rowscaled_wgrad(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                       const float* a_outer, const uint8_t* b,
                                       const uint8_t* b_scales, const float* b_outer,
                                       const int64_t* padded_offsets, int64_t col_rows_cap,
                                       int64_t n, int64_t k, void* out, int out_dtype,
                                       uint32_t* dev_status, void* stream) {
  return nv_wgrad_impl("grouped_gemm_nvfp4_rowscaled_wgrad", G, a, a_scales, a_outer, b, b_scales,
                       b_outer, padded_offsets, col_rows_cap, n, k, out, out_dtype, false,
                       dev_status, stream);
}

int grouped_gemm_nvfp4_rowscaled_wgrad_ex(int64_t G, const uint8_t* a, const uint8_t* a_scales,
                                          const float* a_outer, const uint8_t* b,
                                          const uint8_t* b_scales, const float* b_outer,
                                          const int64_t* padded_offsets, int64_t col_rows_cap,
                                          int64_t n, int64_t k, void* out, int out_dtype,
                                          int accumulate, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_gemm_nvfp4_rowscaled_wgrad_ex";
  if (accumulate != 0 && accumulate != 1)
    return fail(BSG_ERR_UNSUPPORTED, "%s: accumulate must be 0 or 1", fn);
  return nv_wgrad_impl(fn, G, a, a_scales, a_outer, b, b_scales, b_outer, padded_offsets,
                       col_rows_cap, n, k, out, out_dtype, accumulate == 1, dev_status, stream);
}

namespace {

constexpr int64_t kMaxRowStride = (int64_t)1 << 20;  // elements: a tile's rows stay in 31 bits

bool row_stride_ok(int64_t ld, int64_t cols) {
  return ld >= cols && ld % 8 == 0 && ld <= kMaxRowStride;
}

// At most this many output tiles of the smallest kind keep a tile's index in 31 bits.
bool tiles_ok(bool wgrad, int64_t G, int64_t rows_cap, int64_t n, int64_t k) {
  return (wgrad ? G * ((n + 63) / 64) * ((k + 63) / 64)
                : ((rows_cap + 15) / 16 + G) * ((n + 63) / 64)) < ((int64_t)1 << 31);
}

// Whether some call takes these sizes.
bool sizes_16bit_ok(bool wgrad, int64_t G, int64_t rows_cap, int64_t n, int64_t k) {
  return G >= 1 && G <= BSG_MAX_GROUPS && rows_cap >= 0 && rows_cap < ((int64_t)1 << 31) &&
         n > 0 && row_stride_ok(n, n) && k > 0 && row_stride_ok(k, k) &&
         tiles_ok(wgrad, G, rows_cap, n, k);
}

int check_16bit_types(const char* fn, int in_dtype, int out_dtype) {
  if (in_dtype != BSG_IN_BF16 && in_dtype != BSG_IN_F16)
    return fail(BSG_ERR_UNSUPPORTED, "%s: in_dtype %d", fn, in_dtype);
  const int same = in_dtype == BSG_IN_F16 ? BSG_OUT_F16 : BSG_OUT_BF16;
  if (out_dtype != same && out_dtype != BSG_OUT_F32)
    return fail(BSG_ERR_UNSUPPORTED, "%s: out_dtype %d is neither the operands' type nor float32",
                fn, out_dtype);
  return BSG_OK;
}

int check_16bit_workspace(const char* fn, const void* workspace, size_t have, size_t need) {
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(BSG_ERR_ALIGN, "%s: workspace must be 256-byte aligned", fn);
  if (have < need)
    return fail(BSG_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, have, need);
  return BSG_OK;
}

}  // namespace

size_t grouped_gemm_16bit_workspace_size(void) { return bsg::gemm_16bit_workspace_bytes(); }

int grouped_gemm_16bit_tile_rows(int mode, int64_t G, int64_t rows_cap, int64_t n, int64_t k,
                                 int with_workspace) {
  if (mode != BSG_FPROP_TN && mode != BSG_WGRAD_NT && mode != BSG_DGRAD_NN) return 0;
  if (!sizes_16bit_ok(mode == BSG_WGRAD_NT, G, rows_cap, n, k)) return 0;
  return bsg::gemm_16bit_tile_rows(mode, G, rows_cap, n, k, with_workspace != 0);
}

int grouped_gemm_16bit(int mode, int in_dtype, int64_t G, const void* a, int64_t lda,
                       const void* b, int64_t ldb, int64_t stride_b, const int64_t* offsets,
                       int64_t rows_cap, int64_t n, int64_t k, const void* c, void* out,
                       int64_t ldo, int64_t stride_o, int out_dtype, void* workspace,
                       size_t workspace_bytes, uint32_t* dev_status, void* stream) {
  const char* fn = "grouped_gemm_16bit";
  if (a == nullptr || b == nullptr || offsets == nullptr || out == nullptr)
    return fail(BSG_ERR_NULL, "%s: a, b, offsets and out must be non-NULL", fn);
  if (mode != BSG_FPROP_TN && mode != BSG_WGRAD_NT && mode != BSG_DGRAD_NN)
    return fail(BSG_ERR_UNSUPPORTED, "%s: mode %d", fn, mode);
  const int tc = check_16bit_types(fn, in_dtype, out_dtype);
  if (tc != BSG_OK) return tc;
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || rows_cap >= ((int64_t)1 << 31) || n <= 0 || k <= 0 || n % 8 != 0 || k % 8 != 0)
    return fail(BSG_ERR_SHAPE,
                "%s: need 0 <= rows_cap < 2^31 and n, k positive multiples of 8 (got %lld, %lld, %lld)",
                fn, (long long)rows_cap, (long long)n, (long long)k);
  const bool wgrad = mode == BSG_WGRAD_NT;
  const int64_t acols = wgrad ? n : k, bcols = mode == BSG_DGRAD_NN ? n : k;
  const int64_t ocols = wgrad ? k : n;
  if (!row_stride_ok(lda, acols) || !row_stride_ok(ldb, bcols) || !row_stride_ok(ldo, ocols))
    return fail(BSG_ERR_SHAPE,
                "%s: lda=%lld, ldb=%lld, ldo=%lld must be multiples of 8 in [row length, %lld]", fn,
                (long long)lda, (long long)ldb, (long long)ldo, (long long)kMaxRowStride);
  const int64_t brows = mode == BSG_DGRAD_NN ? k : n;
  if (!wgrad && G > 1 && (stride_b % 8 != 0 || stride_b < (brows - 1) * ldb + bcols))
    return fail(BSG_ERR_SHAPE, "%s: stride_b=%lld overlaps the groups or is no multiple of 8", fn,
                (long long)stride_b);
  if (wgrad && G > 1 && (stride_o % 8 != 0 || stride_o < (n - 1) * ldo + k))
    return fail(BSG_ERR_SHAPE, "%s: stride_o=%lld overlaps the groups or is no multiple of 8", fn,
                (long long)stride_o);
  if (!tiles_ok(wgrad, G, rows_cap, n, k))
    return fail(BSG_ERR_SHAPE, "%s: too many output tiles", fn);
  if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned16(c))
    return fail(BSG_ERR_ALIGN, "%s: a, b, c and out must be 16-byte aligned", fn);
  if (workspace != nullptr) {
    const int wc = check_16bit_workspace(fn, workspace, workspace_bytes,
                                         bsg::gemm_16bit_workspace_bytes());
    if (wc != BSG_OK) return wc;
  }
  return hip_result(bsg::launch_gemm_16bit(mode, in_dtype == BSG_IN_F16, (int)G, a, lda, b, ldb,
                                           stride_b, offsets, rows_cap, n, k, c, out, ldo, stride_o,
                                           out_dtype == BSG_OUT_F32, workspace, dev_status,
                                           (hipStream_t)stream),
                    fn);
}

size_t grouped_lora_gemm_16bit_workspace_size(int64_t rows_cap, int64_t n, int64_t k, int64_t rank) {
  if (rows_cap < 0 || n < 0 || k < 0 || rank < 0 || rank > BSG_MAX_LORA_RANK) return 0;
  return bsg::lora_gemm_16bit_workspace_bytes(rows_cap, rank);
}

int grouped_lora_gemm_16bit_tile_rows(int64_t rows_cap, int64_t n, int64_t k) {
  if (!sizes_16bit_ok(false, 1, rows_cap, n, k)) return 0;
  return bsg::lora_gemm_16bit_tile_rows(rows_cap, n, k);
}

int grouped_lora_gemm_16bit(int in_dtype, int64_t G, const void* x, int64_t ldx, const void* w,
                            int64_t ldw, const void* lora_a, const void* lora_b,
                            int64_t num_adapters, int64_t rank, const int64_t* offsets,
                            const int32_t* adapter, const float* scale, int64_t rows_cap,
                            int64_t n, int64_t k, void* out, int64_t ldo, int out_dtype,
                            void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                            void* stream) {
  const char* fn = "grouped_lora_gemm_16bit";
  if (x == nullptr || w == nullptr || lora_a == nullptr || lora_b == nullptr || offsets == nullptr ||
      adapter == nullptr || scale == nullptr || out == nullptr || workspace == nullptr)
    return fail(BSG_ERR_NULL, "%s: every buffer but dev_status must be non-NULL", fn);
  const int tc = check_16bit_types(fn, in_dtype, out_dtype);
  if (tc != BSG_OK) return tc;
  if (G < 1 || G > BSG_MAX_GROUPS)
    return fail(BSG_ERR_SHAPE, "%s: G=%lld outside [1, %d]", fn, (long long)G, BSG_MAX_GROUPS);
  if (rows_cap < 0 || rows_cap >= ((int64_t)1 << 31) || n <= 0 || k <= 0 || n % 8 != 0 || k % 8 != 0)
    return fail(BSG_ERR_SHAPE,
                "%s: need 0 <= rows_cap < 2^31 and n, k positive multiples of 8 (got %lld, %lld, %lld)",
                fn, (long long)rows_cap, (long long)n, (long long)k);
  if (rank < 8 || rank > BSG_MAX_LORA_RANK || rank % 8 != 0)
    return fail(BSG_ERR_SHAPE, "%s: rank=%lld is no multiple of 8 in [8, %d]", fn, (long long)rank,
                BSG_MAX_LORA_RANK);
  if (num_adapters < 1 || num_adapters >= ((int64_t)1 << 31))
    return fail(BSG_ERR_SHAPE, "%s: num_adapters=%lld", fn, (long long)num_adapters);
  if (!row_stride_ok(ldx, k) || !row_stride_ok(ldw, k) || !row_stride_ok(ldo, n))
    return fail(BSG_ERR_SHAPE,
                "%s: ldx=%lld, ldw=%lld, ldo=%lld must be multiples of 8 in [row length, %lld]", fn,
                (long long)ldx, (long long)ldw, (long long)ldo, (long long)kMaxRowStride);
  if (!tiles_ok(false, 1, rows_cap, n, k))
    return fail(BSG_ERR_SHAPE, "%s: too many output tiles", fn);
  if (!aligned16(x) || !aligned16(w) || !aligned16(lora_a) || !aligned16(lora_b) || !aligned16(out))
    return fail(BSG_ERR_ALIGN, "%s: x, w, lora_a, lora_b and out must be 16-byte aligned", fn);
  if (!aligned4(adapter) || !aligned4(scale))
    return fail(BSG_ERR_ALIGN, "%s: adapter and scale must be 4-byte aligned", fn);
  const int wc = check_16bit_workspace(
      fn, workspace, workspace_bytes, bsg::lora_gemm_16bit_workspace_bytes(rows_cap, rank));
  if (wc != BSG_OK) return wc;
  return hip_result(
      bsg::launch_lora_gemm_16bit(in_dtype == BSG_IN_F16, (int)G, x, ldx, w, ldw, lora_a, lora_b,
                                  num_adapters, rank, offsets, adapter, scale, rows_cap, n, k, out,
                                  ldo, out_dtype == BSG_OUT_F32, workspace, dev_status,
                                  (hipStream_t)stream),
      fn);
}

namespace {

size_t grad_elem_bytes(int32_t dtype) { return dtype == BSG_GRAD_F32 ? 4 : 2; }

// Whether a tensor is written while another one, or another part of the same, is read or
// written: workgroups would race.  Returns its index, or -1.  The table that is about to be
// filled serves as scratch: a record for each tensor that holds elements, by its output.
int64_t find_overlap(const void* const* src, void* const* dst, const int64_t* numels,
                     const int32_t* dtypes, bsg::GradChunk* rec, int32_t count) {
  const auto bytes = [&](int32_t i) { return (uintptr_t)numels[i] * grad_elem_bytes(dtypes[i]); };
  const auto begin = [](const bsg::GradChunk& r) { return reinterpret_cast<uintptr_t>(r.dst); };
  int64_t used = 0;
  for (int32_t i = 0; i < count; ++i)
    if (numels[i] != 0) rec[used++] = bsg::GradChunk{src[i], dst[i], i, 0};
  std::sort(rec, rec + used,
            [&](const bsg::GradChunk& a, const bsg::GradChunk& b) { return begin(a) < begin(b); });
  for (int64_t r = 1; r < used; ++r)
    if (begin(rec[r]) < begin(rec[r - 1]) + bytes(rec[r - 1].n)) return rec[r].n;
  for (int32_t i = 0; i < count; ++i) {
    if (numels[i] == 0) continue;
    // the last output that begins before the input's end: where none, or this tensor's own in
    // the same place, no other reaches into the input
    const uintptr_t s = reinterpret_cast<uintptr_t>(src[i]);
    const bsg::GradChunk* after =
        std::lower_bound(rec, rec + used, s + bytes(i),
                         [&](const bsg::GradChunk& r, uintptr_t end) { return begin(r) < end; });
    if (after == rec) continue;
    const bsg::GradChunk& d = after[-1];
    if (begin(d) + bytes(d.n) > s && !(d.n == i && begin(d) == s)) return i;
  }
  return -1;
}

}  // namespace

int grad_clip_plan_fill(int64_t num_tensors, const void* const* src, void* const* dst,
                        const int64_t* numels, const int32_t* dtypes, void* plan,
                        size_t plan_bytes, int64_t* num_chunks) {
  const char* fn = "grad_clip_plan_fill";
  if (num_chunks == nullptr || src == nullptr || dst == nullptr || numels == nullptr ||
      dtypes == nullptr)
    return fail(BSG_ERR_NULL, "%s: src, dst, numels, dtypes and num_chunks must be non-NULL", fn);
  if (num_tensors < 0 || num_tensors >= ((int64_t)1 << 31))
    return fail(BSG_ERR_SHAPE, "%s: num_tensors=%lld", fn, (long long)num_tensors);
  bsg::GradChunk* out = static_cast<bsg::GradChunk*>(plan);
  const int64_t room = plan != nullptr ? (int64_t)(plan_bytes / sizeof(bsg::GradChunk)) : 0;
  // the first chunk is as much shorter as puts the later ones on 128-byte lines
  const auto first_chunk = [&](int64_t i) {
    return bsg::kGradChunk - (int64_t)(reinterpret_cast<uintptr_t>(src[i]) % 128 /
                                       grad_elem_bytes(dtypes[i]));
  };
  int64_t count = 0;
  for (int64_t i = 0; i < num_tensors; ++i) {
    if (dtypes[i] != BSG_GRAD_BF16 && dtypes[i] != BSG_GRAD_F16 && dtypes[i] != BSG_GRAD_F32)
      return fail(BSG_ERR_UNSUPPORTED, "%s: tensor %lld has dtype %d", fn, (long long)i, dtypes[i]);
    if (numels[i] < 0 || numels[i] >= ((int64_t)1 << 48))
      return fail(BSG_ERR_SHAPE, "%s: tensor %lld has %lld elements", fn, (long long)i,
                  (long long)numels[i]);
    if (numels[i] == 0) continue;
    if (src[i] == nullptr || dst[i] == nullptr)
      return fail(BSG_ERR_NULL, "%s: tensor %lld has no data", fn, (long long)i);
    const uintptr_t esz = grad_elem_bytes(dtypes[i]);
    if (reinterpret_cast<uintptr_t>(src[i]) % esz != 0 || reinterpret_cast<uintptr_t>(dst[i]) % esz != 0)
      return fail(BSG_ERR_ALIGN, "%s: tensor %lld is not aligned to its elements", fn, (long long)i);
    const int64_t rest = numels[i] - first_chunk(i);
    count += 1 + (rest > 0 ? (rest + bsg::kGradChunk - 1) / bsg::kGradChunk : 0);
  }
  if (plan != nullptr) {
    if (count > room)
      return fail(BSG_ERR_WORKSPACE, "%s: a plan of %zu bytes is too small", fn, plan_bytes);
    const int64_t bad = find_overlap(src, dst, numels, dtypes, out, (int32_t)num_tensors);
    if (bad >= 0)
      return fail(BSG_ERR_SHAPE, "%s: tensor %lld shares memory with another one's output, or in "
                  "part with its own", fn, (long long)bad);
    for (int64_t i = 0; i < num_tensors; ++i) {
      const uintptr_t esz = grad_elem_bytes(dtypes[i]);
      int64_t take = first_chunk(i);
      for (int64_t at = 0; at < numels[i]; at += take, take = bsg::kGradChunk) {
        if (take > numels[i] - at) take = numels[i] - at;
        *out++ = bsg::GradChunk{static_cast<const char*>(src[i]) + (uintptr_t)at * esz,
                                static_cast<char*>(dst[i]) + (uintptr_t)at * esz, (int32_t)take,
                                dtypes[i]};
      }
    }
  }
  *num_chunks = count;
  return ok();
}

size_t grad_clip_workspace_size(void) { return sizeof(double) * bsg::kGradMaxBlocks; }

namespace {

int check_grad_call(const char* fn, const void* plan, int64_t num_chunks, const void* workspace,
                    size_t workspace_bytes) {
  if (workspace == nullptr || (plan == nullptr && num_chunks != 0))
    return fail(BSG_ERR_NULL, "%s: plan and workspace must be non-NULL", fn);
  if (num_chunks < 0) return fail(BSG_ERR_SHAPE, "%s: num_chunks=%lld", fn, (long long)num_chunks);
  if (((reinterpret_cast<uintptr_t>(plan) | reinterpret_cast<uintptr_t>(workspace)) & 7u) != 0)
    return fail(BSG_ERR_ALIGN, "%s: plan and workspace must be 8-byte aligned", fn);
  if (workspace_bytes < grad_clip_workspace_size())
    return fail(BSG_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes,
                grad_clip_workspace_size());
  return BSG_OK;
}

}  // namespace

int grad_norm(const void* plan, int64_t num_chunks, void* workspace, size_t workspace_bytes,
              float* norm, double* sumsq, uint32_t* dev_status, void* stream) {
  const char* fn = "grad_norm";
  const int cc = check_grad_call(fn, plan, num_chunks, workspace, workspace_bytes);
  if (cc != BSG_OK) return cc;
  if (norm == nullptr && sumsq == nullptr)
    return fail(BSG_ERR_NULL, "%s: no output requested", fn);
  if (!aligned4(norm) || (reinterpret_cast<uintptr_t>(sumsq) & 7u) != 0)
    return fail(BSG_ERR_ALIGN, "%s: norm must be 4-byte and sumsq 8-byte aligned", fn);
  return hip_result(bsg::launch_grad_norm(static_cast<const bsg::GradChunk*>(plan), num_chunks,
                                          static_cast<double*>(workspace), norm, sumsq, dev_status,
                                          (hipStream_t)stream),
                    fn);
}

int clip_grad_norm(const void* plan, int64_t num_chunks, float max_norm, const double* sumsq,
                   void* workspace, size_t workspace_bytes, float* norm, uint32_t* dev_status,
                   void* stream) {
  const char* fn = "clip_grad_norm";
  const int cc = check_grad_call(fn, plan, num_chunks, workspace, workspace_bytes);
  if (cc != BSG_OK) return cc;
  if (!(max_norm >= 0.0f))
    return fail(BSG_ERR_SHAPE, "%s: max_norm=%g must be >= 0", fn, (double)max_norm);
  if (!aligned4(norm) || (reinterpret_cast<uintptr_t>(sumsq) & 7u) != 0)
    return fail(BSG_ERR_ALIGN, "%s: norm must be 4-byte and sumsq 8-byte aligned", fn);
  return hip_result(bsg::launch_clip_grad_norm(static_cast<const bsg::GradChunk*>(plan), num_chunks,
                                               max_norm, sumsq, static_cast<double*>(workspace),
                                               norm, dev_status, (hipStream_t)stream),
                    fn);
}

}  // extern "C"
