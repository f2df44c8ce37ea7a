// 16-bit grouped products, large form: the launchers.
#include "gemm_large.h"

namespace bsg {
namespace g16 {

namespace {

template <bool F16>
hipError_t launch_mode(int mode, const Args& p, hipStream_t stream) {
  if (mode == kFprop) return large::launch<kFprop, F16>(p, stream);
  if (mode == kWgrad) return large::launch<kWgrad, F16>(p, stream);
  if (mode == kDgrad) return large::launch<kDgrad, F16>(p, stream);
  return large::launch<kLora, F16>(p, stream);
}

}  // namespace

hipError_t launch_large(int mode, int f16, const Args& p, hipStream_t stream) {
  return f16 ? launch_mode<true>(mode, p, stream) : launch_mode<false>(mode, p, stream);
}

size_t large_workspace_bytes() {
  return (size_t)kWsHeader + (size_t)device_cu_count() * (size_t)large::kPartBytes;
}

}  // namespace g16
}  // namespace bsg
