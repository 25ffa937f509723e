// Launcher of the gated product on block-scaled FP8 operands.
#include "stream_kernel.h"
#include "tile_kernel.h"

namespace fp8q {

template <int OUT>
static hipError_t go(const FfnArgs& p, hipStream_t st) {
  return streams(true, p.M, p.N) ? launch_stream<false, true, OUT>(p, st) : launch_tile<false, true, OUT>(p, st);
}

hipError_t launch_fp8_gated(const FfnArgs& p, bool out_bf16, hipStream_t st) {
  return out_bf16 ? go<kOutBF16>(p, st) : go<kOutF32>(p, st);
}

}  // namespace fp8q
