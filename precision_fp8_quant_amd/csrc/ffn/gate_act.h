// The gate's activation and its slope, shared by the forward and backward
// kernels of the gated feed-forward block.
//
// Both activations are g * sigma(t(g)), sigma(t) = 1 / (1 + e^-t), with
//   t(g) = g (c1 + c3 g^2)
//   SiLU:      c1 = 1,              c3 = 0
//   GELU-tanh: c1 = 2 sqrt(2 / pi), c3 = 0.044715 c1
//              (0.5 (1 + tanh z) = sigma(2 z))
// so one code path serves both and the choice is two kernel arguments.
//   act(g)  = g s,                             s = sigma(t)
//   act'(g) = s + g s (1 - s) t'(g),           t'(g) = c1 + 3 c3 g^2
#pragma once

#include <hip/hip_runtime.h>

namespace fp8q {

// act(g) * u.  e = exp(-|t|) is at most 1, so neither 1 + e nor its reciprocal
// can overflow; sigma is r or e r.  v_exp_f32 of the rounded product
// |t| log2(e) is off by about |t| 2^-24 in relative terms, which weighs
// e / (1 + e) in sigma.  g^2 is held at 1e4 (|g| = 100, where sigma has long
// been 0 or 1 for both activations), so that it cannot overflow into 0 * inf.
__device__ __forceinline__ float gate_mul(float g, float u, float c1, float c3) {
  const float t = g * __builtin_fmaf(c3, __builtin_fminf(g * g, 1.0e4f), c1);
  const float e = __builtin_amdgcn_exp2f(-1.44269504088896341f * __builtin_fabsf(t));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  return g * (t >= 0.0f ? r : e * r) * u;
}

}  // namespace fp8q
