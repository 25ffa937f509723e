// Launchers of the 8-bit integer products.
#include "stream_kernel.h"

namespace fp8q {

hipError_t launch_int8_gemm(const FfnArgs& p, bool out_bf16, hipStream_t st) {
  return out_bf16 ? launch_stream<true, false, kOutBF16>(p, st) : launch_stream<true, false, kOutF32>(p, st);
}

hipError_t launch_int8_gated(const FfnArgs& p, bool out_bf16, hipStream_t st) {
  return out_bf16 ? launch_stream<true, true, kOutBF16>(p, st) : launch_stream<true, true, kOutF32>(p, st);
}

}  // namespace fp8q
