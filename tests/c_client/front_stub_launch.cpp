// Host-only stand-ins for the launchers behind include/fp8q_front.h, so that
// abi_front.cpp can be built and run without a GPU under the host sanitizers.
// Each stub only counts its calls.
#include "front/front_launch.h"

extern "C" {
int fp8q_front_stub_launches = 0;
}

namespace fp8q {

static hipError_t hit() {
  ++fp8q_front_stub_launches;
  return hipSuccess;
}

hipError_t launch_fp8_rmsnorm(const NormArgs&, bool, bool, int, hipStream_t) { return hit(); }
hipError_t launch_int8_rmsnorm(const NormArgs&, bool, bool, hipStream_t) { return hit(); }
hipError_t launch_rmsnorm_backward(const NormBwdArgs&, bool, bool, hipStream_t) { return hit(); }
hipError_t launch_moe_route(const RouteArgs&, bool, hipStream_t) { return hit(); }
hipError_t launch_moe_route_backward(const RouteBwdArgs&, bool, hipStream_t) { return hit(); }
hipError_t launch_moe_dispatch(const DispatchArgs&, hipStream_t) { return hit(); }

}  // namespace fp8q
