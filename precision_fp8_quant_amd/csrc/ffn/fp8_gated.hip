// Launcher of the gated product on block-scaled FP8 operands.
#include "stream_kernel.h"

namespace fp8q {

hipError_t launch_fp8_gated(const FfnArgs& p, bool out_bf16, hipStream_t st) {
  return out_bf16 ? launch_stream<false, true, kOutBF16>(p, st) : launch_stream<false, true, kOutF32>(p, st);
}

}  // namespace fp8q
