// Internal launchers behind include/fp8q_ffn.h.  Arguments are validated by
// abi_ffn.cpp before any of these is called; each enqueues on `st` and returns
// the launch status without synchronising.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fp8q {

// HIP takes launches of fewer than 2^32 threads.
constexpr int64_t max_grid(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

// Workgroups for `units` of them: kernels with a loop over the grid do what is left in further rounds.
inline unsigned grid_of(int64_t units, int threads) {
  return unsigned(units < max_grid(threads) ? units : max_grid(threads));
}

// One product (or gated pair of products) of K-contiguous 8-bit operands.
struct FfnArgs {
  const uint8_t* a; int64_t lda; const float* sa;
  const uint8_t* b; int64_t ldb; const float* sb;
  const float* bias;              // FP32 [N] or nullptr (plain product)
  void* c; int64_t ldc;           // C[M][N], or h[M][F]
  void* gu; int64_t ldgu;         // gate and up before the activation, or nullptr
  int64_t M, N, K;                // N: columns of c (F where the product is gated)
  int64_t up;                     // gated: rows of b (scales, columns of gu) from the gate's to the up's
  float act_c1, act_c3;           // the activation's sigma argument (gate_act.h)
};

hipError_t launch_fp8_gated(const FfnArgs& p, bool out_bf16, hipStream_t st);
hipError_t launch_int8_gemm(const FfnArgs& p, bool out_bf16, hipStream_t st);
hipError_t launch_int8_gated(const FfnArgs& p, bool out_bf16, hipStream_t st);

hipError_t launch_gated_backward(float act_c1, float act_c3, int64_t M, int64_t F, const void* dh, int64_t ld_dh,
                                 const void* gu, int64_t ld_gu, bool bf16, int mode, uint8_t* q, int64_t ld_q,
                                 float* scales, uint8_t* q_t, int64_t ld_qt, float* scales_t, void* dgu,
                                 int64_t ld_dgu, hipStream_t st);

hipError_t launch_int8_quant_rows(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q,
                                  int64_t ld_q, float* scales, hipStream_t st);

}  // namespace fp8q
