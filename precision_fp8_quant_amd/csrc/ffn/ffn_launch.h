// Internal launchers behind include/fp8q_ffn.h.  Arguments are validated by
// abi_ffn.cpp before any of these is called; each enqueues on `st` and returns
// the launch status without synchronising.
#pragma once

#include "launch_plan.h"

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fp8q {

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
  int64_t sa_ld;                  // FP8: scales of A from one K-group to the next
};

// Rows [m0, m0 + rows) and columns [n0, n0 + cols) of a product; n0 in whole 128 columns where the operands are FP8.
inline FfnArgs part_of(const FfnArgs& p, bool int8, bool out_bf16, int64_t m0, int64_t rows, int64_t n0, int64_t cols) {
  const int64_t es = out_bf16 ? 2 : 4;
  FfnArgs q = p;
  q.M = rows;
  q.N = cols;
  if (p.K > 0) {                  // otherwise there may be no operands
    q.a = p.a + m0 * p.lda;
    q.sa = p.sa + m0;
    q.b = p.b + n0 * p.ldb;
    q.sb = p.sb + (int8 ? n0 : n0 / 128 * ((p.K + 127) / 128));
  }
  if (p.bias) q.bias = p.bias + n0;
  q.c = static_cast<uint8_t*>(p.c) + (m0 * p.ldc + n0) * es;
  if (p.gu) q.gu = static_cast<uint8_t*>(p.gu) + (m0 * p.ldgu + n0) * es;
  return q;
}

// launch(part, workgroups) for the whole product in tiles of bm x bn, as many times as the grid's limit asks for.
template <typename Launch>
hipError_t in_pieces(const FfnArgs& p, bool int8, bool out_bf16, int64_t bm, int64_t bn, int threads, Launch launch) {
  const Piece s = piece_size(p.M, p.N, bm, bn, threads);
  for (int64_t m0 = 0; m0 < p.M; m0 += s.rows)
    for (int64_t n0 = 0; n0 < p.N; n0 += s.cols) {
      const int64_t rows = p.M - m0 < s.rows ? p.M - m0 : s.rows, cols = p.N - n0 < s.cols ? p.N - n0 : s.cols;
      const hipError_t e = launch(part_of(p, int8, out_bf16, m0, rows, n0, cols),
                                  unsigned(((rows + bm - 1) / bm) * ((cols + bn - 1) / bn)));
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

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
