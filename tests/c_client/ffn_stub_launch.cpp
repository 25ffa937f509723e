// Host-only stand-ins for the launchers behind include/fp8q_ffn.h, so that
// abi_ffn.cpp can be built and run without a GPU under the host sanitizers.
// Each stub only counts its calls.
#include "ffn/ffn_launch.h"

extern "C" {
int fp8q_ffn_stub_launches = 0;
}

namespace fp8q {

static hipError_t hit() {
  ++fp8q_ffn_stub_launches;
  return hipSuccess;
}

hipError_t launch_fp8_gated(const FfnArgs&, bool, hipStream_t) { return hit(); }
hipError_t launch_int8_gemm(const FfnArgs&, bool, hipStream_t) { return hit(); }
hipError_t launch_int8_gated(const FfnArgs&, bool, hipStream_t) { return hit(); }
hipError_t launch_gated_backward(float, float, int64_t, int64_t, const void*, int64_t, const void*, int64_t, bool, int,
                                 uint8_t*, int64_t, float*, uint8_t*, int64_t, float*, void*, int64_t, hipStream_t) {
  return hit();
}
hipError_t launch_int8_quant_rows(const void*, bool, int64_t, int64_t, int64_t, int8_t*, int64_t, float*, hipStream_t) {
  return hit();
}

}  // namespace fp8q
