// Launchers of the 8-bit integer products.
#include "stream_kernel.h"
#include "tile_kernel.h"

namespace fp8q {

template <bool GATED, int OUT>
static hipError_t go(const FfnArgs& p, hipStream_t st) {
  return streams(GATED, p.M, p.N) ? launch_stream<true, GATED, OUT>(p, st) : launch_tile<true, GATED, OUT>(p, st);
}

hipError_t launch_int8_gemm(const FfnArgs& p, bool out_bf16, hipStream_t st) {
  return out_bf16 ? go<false, kOutBF16>(p, st) : go<false, kOutF32>(p, st);
}

hipError_t launch_int8_gated(const FfnArgs& p, bool out_bf16, hipStream_t st) {
  return out_bf16 ? go<true, kOutBF16>(p, st) : go<true, kOutF32>(p, st);
}

}  // namespace fp8q
