// 16-bit grouped products, small form: the launchers.
#include "gemm_small.h"

namespace bsg {
namespace g16 {

namespace {

template <bool F16, int BM>
hipError_t launch_mode(int mode, const Args& p, hipStream_t stream) {
  if (mode == kFprop) return small::launch<kFprop, F16, BM>(p, stream);
  if (mode == kDgrad) return small::launch<kDgrad, F16, BM>(p, stream);
  if (mode == kLora) return small::launch<kLora, F16, BM>(p, stream);
  return small::launch<kWgrad, F16, 128>(p, stream);
}

template <bool F16>
hipError_t launch_bm(int mode, int bm, const Args& p, hipStream_t stream) {
  if (bm <= 32) return launch_mode<F16, 32>(mode, p, stream);
  if (bm <= 64) return launch_mode<F16, 64>(mode, p, stream);
  return launch_mode<F16, 128>(mode, p, stream);
}

}  // namespace

hipError_t launch_small(int mode, int f16, int bm, const Args& p, hipStream_t stream) {
  return f16 ? launch_bm<true>(mode, bm, p, stream) : launch_bm<false>(mode, bm, p, stream);
}

size_t small_workspace_bytes() {
  return (size_t)kWsHeader +
         (size_t)(small::kWgPerCu * device_cu_count()) * (size_t)small::kPartBytes<128>;
}

}  // namespace g16
}  // namespace bsg
