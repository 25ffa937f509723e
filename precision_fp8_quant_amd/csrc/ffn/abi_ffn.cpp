// C ABI of the gated feed-forward operators (include/fp8q_ffn.h): argument
// validation, then dispatch to the HIP launchers.  Every check runs on the
// host before anything is enqueued; the first violation returns its status
// and nothing is launched.
#include "../../../include/fp8q_ffn.h"
#include "../abi_check.hpp"
#include "ffn_launch.h"

#include <stdint.h>

namespace {

// The largest K whose 8-bit sum fits 32 bits: 128 * 128 * 131056 < 2^31.
constexpr int64_t kMaxInt8K = 131056;

bool act_ok(int act) { return act == FP8Q_ACT_SILU || act == FP8Q_ACT_GELU_TANH; }

// Coefficients of the activation's sigma argument (ffn/gate_act.h).
void set_act(int act, float* c1, float* c3) {
  const double c = 1.59576912160573071176;   // 2 sqrt(2 / pi)
  *c1 = act == FP8Q_ACT_SILU ? 1.0f : float(c);
  *c3 = act == FP8Q_ACT_SILU ? 0.0f : float(0.044715 * c);
}

bool round_up(int64_t x, int64_t to, int64_t* out) {
  if (__builtin_add_overflow(x, to - 1, out)) return false;
  *out -= *out % to;
  return true;
}

// Every pair of outputs and every output against every input.
template <int NO, int NI>
int check_ranges(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int i = 0; i < NO; ++i)
    if (!outs[i].ok) return FP8Q_ERR_SHAPE;
  for (int i = 0; i < NI; ++i)
    if (!ins[i].ok) return FP8Q_ERR_SHAPE;
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return FP8Q_ERR_ALIAS;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return FP8Q_ERR_ALIAS;
  }
  return FP8Q_OK;
}

// More outputs than a card's memory holds, as 16 x 16 tiles: up to here sizes and tile numbers stay far from overflow.
// (Products of more tiles than one launch takes are cut up, ffn_launch.h.)
bool grid_ok(int64_t M, int64_t N) {
  const int64_t tm = (M - 1) / 16 + 1, tn = (N - 1) / 16 + 1;
  return tn <= kMaxGridX / tm;
}

// Shared by the two integer products: b has `brows` rows, c is [M][N].
int check_int8(int64_t M, int64_t N, int64_t K, int64_t brows, const int8_t* a, int64_t lda, const float* sa,
               const int8_t* b, int64_t ldb, const float* sb, const float* bias, void* c, int c_dtype,
               int64_t ldc) {
  if (!c) return FP8Q_ERR_NULL;
  if (K > 0 && (!a || !b || !sa || !sb)) return FP8Q_ERR_NULL;
  if (ldc < N || (K > 0 && (lda < K || ldb < K))) return FP8Q_ERR_SHAPE;
  const int64_t es = dtype_size(c_dtype);
  if (!aligned16(c) || !ld16(ldc, es) || (bias && !aligned16(bias))) return FP8Q_ERR_ALIGN;
  if (K > 0 && (!aligned16(a) || !aligned16(b) || !aligned16(sa) || !aligned16(sb) || lda % 16 || ldb % 16))
    return FP8Q_ERR_ALIGN;
  if (K > kMaxInt8K || (K > 0 && (lda > kMaxGemmLd || ldb > kMaxGemmLd)) || !grid_ok(M, N))
    return FP8Q_ERR_UNSUPPORTED;
  const int64_t kr = (K + 15) / 16 * 16;          // what is read of a row
  const bool k0 = K == 0;
  const Range outs[1] = {span(c, M, N, ldc, es)};
  const Range ins[5] = {span(a, k0 ? 0 : M, kr, lda, 1), span(b, k0 ? 0 : brows, kr, ldb, 1),
                        span(sa, k0 ? 0 : 1, M, M, 4), span(sb, k0 ? 0 : 1, brows, brows, 4),
                        span(bias, bias ? 1 : 0, N, N, 4)};
  return check_ranges(outs, ins);
}

}  // namespace

extern "C" {

int fp8_gemm_gated(int act, int64_t M, int64_t F, int64_t K, const uint8_t* a, int64_t lda, const float* a_scales,
                   const uint8_t* b, int64_t ldb, const float* b_scales, void* h, int out_dtype, int64_t ldh,
                   void* gu, int64_t ldgu, void* stream) {
  if (!act_ok(act) || !dtype_ok(out_dtype)) return FP8Q_ERR_ARG;
  if (M < 0 || F < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || F == 0) return FP8Q_OK;
  if (!h) return FP8Q_ERR_NULL;
  if (K > 0 && (!a || !b || !a_scales || !b_scales)) return FP8Q_ERR_NULL;
  int64_t f2 = 0, nsa = 0, nsb = 0;
  if (!mul_ok(F, 2, &f2)) return FP8Q_ERR_SHAPE;
  if (ldh < F || (gu && ldgu < f2) || (K > 0 && (lda < K || ldb < K))) return FP8Q_ERR_SHAPE;
  const int64_t es = dtype_size(out_dtype);
  if (!aligned16(h) || !ld16(ldh, es) || (gu && (!aligned16(gu) || !ld16(ldgu, es)))) return FP8Q_ERR_ALIGN;
  if (K > 0 && (!aligned16(a) || !aligned16(b) || !aligned16(a_scales) || !aligned16(b_scales) || lda % 16 ||
                ldb % 16))
    return FP8Q_ERR_ALIGN;
  if (F % 128 || K % 128) return FP8Q_ERR_UNSUPPORTED;
  if ((K > 0 && (lda > kMaxGemmLd || ldb > kMaxGemmLd)) || !grid_ok(M, F)) return FP8Q_ERR_UNSUPPORTED;
  if (!mul_ok(K / 128, M, &nsa) || !mul_ok(f2 / 128, K / 128, &nsb)) return FP8Q_ERR_SHAPE;
  const bool k0 = K == 0;
  const Range outs[2] = {span(h, M, F, ldh, es), span(gu, gu ? M : 0, f2, ldgu, es)};
  const Range ins[4] = {span(a, M, K, lda, 1), span(b, f2, K, ldb, 1), span(a_scales, k0 ? 0 : 1, nsa, nsa, 4),
                        span(b_scales, k0 ? 0 : 1, nsb, nsb, 4)};
  const int bad = check_ranges(outs, ins);
  if (bad != FP8Q_OK) return bad;
  fp8q::FfnArgs p{a, lda, a_scales, b, ldb, b_scales, nullptr, h, ldh, gu, ldgu, M, F, K, F, 0.0f, 0.0f, M};
  set_act(act, &p.act_c1, &p.act_c3);
  return from_hip(fp8q::launch_fp8_gated(p, out_dtype == FP8Q_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_gated_backward(int act, int64_t M, int64_t F, const void* dh, int64_t ld_dh, const void* gu, int64_t ld_gu,
                       int x_dtype, int mode, uint8_t* q, int64_t ld_q, float* scales, uint8_t* q_t, int64_t ld_qt,
                       float* scales_t, void* dgu, int64_t ld_dgu, void* stream) {
  if (!act_ok(act) || !dtype_ok(x_dtype)) return FP8Q_ERR_ARG;
  if (mode != FP8Q_SCALE_MAXABS && mode != FP8Q_SCALE_POW2) return FP8Q_ERR_ARG;
  if (M < 0 || F < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || F == 0) return FP8Q_OK;
  if (!dh || !gu || !q || !scales || !q_t || !scales_t) return FP8Q_ERR_NULL;
  int64_t f2 = 0, mp = 0, n1 = 0, n2 = 0;
  if (!mul_ok(F, 2, &f2) || !round_up(M, 128, &mp)) return FP8Q_ERR_SHAPE;
  if (ld_dh < F || ld_gu < f2 || ld_q < f2 || ld_qt < mp || (dgu && ld_dgu < f2)) return FP8Q_ERR_SHAPE;
  const int64_t es = dtype_size(x_dtype);
  if (!aligned16(dh) || !aligned16(gu) || !aligned16(q) || !aligned16(scales) || !aligned16(q_t) ||
      !aligned16(scales_t) || !ld16(ld_dh, es) || !ld16(ld_gu, es) || ld_q % 16 || ld_qt % 16 ||
      (dgu && (!aligned16(dgu) || !ld16(ld_dgu, es))))
    return FP8Q_ERR_ALIGN;
  if (F % 128) return FP8Q_ERR_UNSUPPORTED;
  if (!mul_ok(f2 / 128, mp, &n1) || !mul_ok(mp / 128, f2, &n2)) return FP8Q_ERR_SHAPE;
  const Range outs[5] = {span(q, mp, f2, ld_q, 1), span(scales, 1, n1, n1, 4), span(q_t, f2, mp, ld_qt, 1),
                         span(scales_t, 1, n2, n2, 4), span(dgu, dgu ? M : 0, f2, ld_dgu, es)};
  const Range ins[2] = {span(dh, M, F, ld_dh, es), span(gu, M, f2, ld_gu, es)};
  const int bad = check_ranges(outs, ins);
  if (bad != FP8Q_OK) return bad;
  float c1 = 0.0f, c3 = 0.0f;
  set_act(act, &c1, &c3);
  return from_hip(fp8q::launch_gated_backward(c1, c3, M, F, dh, ld_dh, gu, ld_gu, x_dtype == FP8Q_BF16, mode, q,
                                              ld_q, scales, q_t, ld_qt, scales_t, dgu, ld_dgu,
                                              reinterpret_cast<hipStream_t>(stream)));
}

int int8_quant_rows(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q, int64_t ld_q,
                    float* scales, void* stream) {
  if (!dtype_ok(x_dtype)) return FP8Q_ERR_ARG;
  if (rows < 0 || cols < 0) return FP8Q_ERR_SHAPE;
  if (rows == 0) return FP8Q_OK;
  if (!scales || (cols > 0 && (!x || !q))) return FP8Q_ERR_NULL;
  if (cols > 0 && (ld_x < cols || ld_q < cols)) return FP8Q_ERR_SHAPE;
  const int64_t es = dtype_size(x_dtype);
  if (!aligned16(scales) || (cols > 0 && (!aligned16(x) || !aligned16(q) || !ld16(ld_x, es) || ld_q % 16)))
    return FP8Q_ERR_ALIGN;
  const Range outs[2] = {span(q, rows, cols, ld_q, 1), span(scales, 1, rows, rows, 4)};
  const Range ins[1] = {span(x, rows, cols, ld_x, es)};
  const int bad = check_ranges(outs, ins);
  if (bad != FP8Q_OK) return bad;
  return from_hip(fp8q::launch_int8_quant_rows(x, x_dtype == FP8Q_BF16, rows, cols, ld_x, q, ld_q, scales,
                                               reinterpret_cast<hipStream_t>(stream)));
}

int int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a, int64_t lda, const float* a_scales, const int8_t* b,
              int64_t ldb, const float* b_scales, const float* bias, void* c, int c_dtype, int64_t ldc,
              void* stream) {
  if (!dtype_ok(c_dtype)) return FP8Q_ERR_ARG;
  if (M < 0 || N < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || N == 0) return FP8Q_OK;
  const int bad = check_int8(M, N, K, N, a, lda, a_scales, b, ldb, b_scales, bias, c, c_dtype, ldc);
  if (bad != FP8Q_OK) return bad;
  const fp8q::FfnArgs p{reinterpret_cast<const uint8_t*>(a), lda, a_scales, reinterpret_cast<const uint8_t*>(b), ldb,
                        b_scales, bias, c, ldc, nullptr, 0, M, N, K, 0, 0.0f, 0.0f, 0};
  return from_hip(fp8q::launch_int8_gemm(p, c_dtype == FP8Q_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int int8_gemm_gated(int act, int64_t M, int64_t F, int64_t K, const int8_t* a, int64_t lda, const float* a_scales,
                    const int8_t* b, int64_t ldb, const float* b_scales, void* h, int out_dtype, int64_t ldh,
                    void* stream) {
  if (!act_ok(act) || !dtype_ok(out_dtype)) return FP8Q_ERR_ARG;
  if (M < 0 || F < 0 || K < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || F == 0) return FP8Q_OK;
  int64_t f2 = 0;
  if (!mul_ok(F, 2, &f2)) return FP8Q_ERR_SHAPE;
  const int bad = check_int8(M, F, K, f2, a, lda, a_scales, b, ldb, b_scales, nullptr, h, out_dtype, ldh);
  if (bad != FP8Q_OK) return bad;
  fp8q::FfnArgs p{reinterpret_cast<const uint8_t*>(a), lda, a_scales, reinterpret_cast<const uint8_t*>(b), ldb,
                  b_scales, nullptr, h, ldh, nullptr, 0, M, F, K, F, 0.0f, 0.0f, 0};
  set_act(act, &p.act_c1, &p.act_c3);
  return from_hip(fp8q::launch_int8_gated(p, out_dtype == FP8Q_BF16, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
