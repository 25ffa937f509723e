/*
 * fp8q -- operators of the gated feed-forward block for AMD Instinct MI355X
 * (gfx950).  C ABI, exported by the same library as include/fp8q.h.
 *
 *   h = act(x Wg^T) * (x Wu^T)
 *
 * is trained in block-scaled FP8 (fp8_gemm_gated, fp8_gated_backward around
 * the quantizers and GEMMs of fp8q.h) and served in FP8 or in 8-bit integers
 * (int8_quant_rows, int8_gemm, int8_gemm_gated).  The operators here take any
 * number of tokens; fp8_gemm_blockscaled, which does the down projection in
 * FP8, takes rows in whole tiles of 128: let h be the head of a buffer of such
 * tiles whose other rows are zeros, and quantize and multiply the buffer.
 *
 * Every convention of fp8q.h holds here: device pointers owned by the caller,
 * no allocation, no state, no synchronisation, all work on `stream`, plain int
 * status codes and enum values, arguments validated before anything is
 * launched, row-major matrices with leading dimensions in elements, 16-byte
 * aligned pointers and leading dimensions of a multiple of 16 bytes, finite
 * inputs, outputs that overlap neither inputs nor each other.
 *
 * Activations.  Both are g * sigma(t(g)) with sigma(t) = 1 / (1 + e^-t):
 *   FP8Q_ACT_SILU       t = g
 *   FP8Q_ACT_GELU_TANH  t = 2 sqrt(2/pi) (g + 0.044715 g^3), which is
 *                       0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)))
 * evaluated in FP32 from FP32 pre-activations; each output is rounded once.
 *
 * Weights of a gated projection are stacked: rows [0, F) of B are the gate
 * projection, rows [F, 2F) the up projection, each stored [out][in].
 */
#ifndef FP8Q_FFN_H
#define FP8Q_FFN_H

#include "fp8q.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FP8Q_ACT_SILU = 0, FP8Q_ACT_GELU_TANH = 1 } fp8q_act;

/*
 * fp8_gemm_gated -- both projections, the activation and the product in one
 * kernel, from block-scaled FP8 operands:
 *   g[m][f] = sum_k A[m][k] B[f][k],  u[m][f] = sum_k A[m][k] B[F+f][k]
 *   h[m][f] = act(g[m][f]) * u[m][f]
 * with the per-128-K-group scales and FP32 promotion of fp8_gemm_blockscaled
 * (FPROP), and its precision: within a K-group the matrix instruction drops
 * low bits of its partial sums, so that g and u are off by about 1.5e-5 (5e-5
 * where codes fill their range) in relative Frobenius terms -- more than the
 * rounding of an FP32 output, less than that of a BF16 one.
 *
 * a        : A[M][K] E4M3, leading dimension lda (bytes); any M, one token included.
 * a_scales : [K/128][M] packed (fp8_quant_tile, FP8Q_TILE_1x128).
 * b        : B[2F][K] E4M3, leading dimension ldb (bytes): gate rows, then up rows.
 * b_scales : [2F/128][K/128] packed (fp8_quant_block of the stacked weight).
 * h        : h[M][F], leading dimension ldh, dtype out_dtype (FP8Q_BF16 or FP8Q_F32).
 * gu       : optional (NULL to skip): gu[M][2F], leading dimension ldgu, dtype
 *            out_dtype: g in columns [0, F), u in columns [F, 2F), each
 *            rounded once from FP32 -- what fp8_gated_backward takes.  h is
 *            formed from the unrounded g and u.
 * Requires F and K multiples of 128, lda and ldb of at most 4,194,176 bytes,
 * at most 2^31-1 tiles of 16x16 in h (FP8Q_ERR_UNSUPPORTED).  M == 0 or F == 0
 * is a no-op; K == 0 writes zeros.
 */
int fp8_gemm_gated(int act, int64_t M, int64_t F, int64_t K,
                   const uint8_t* a, int64_t lda, const float* a_scales,
                   const uint8_t* b, int64_t ldb, const float* b_scales,
                   void* h, int out_dtype, int64_t ldh,
                   void* gu, int64_t ldgu,
                   void* stream);

/*
 * fp8_gated_backward -- gradient of h = act(g) * u, quantized for both of the
 * GEMMs that take it in the same pass:
 *   dg = dh * u * act'(g),  du = dh * act(g),  D = [dg | du]
 * D is formed in FP32 from the inputs and quantized from FP32 (never rounded
 * to BF16 in between), in 1x128 tiles for Dgrad (dX = D [Wg; Wu]) and in
 * transposed 128x1 tiles for Wgrad (d[Wg; Wu] = D^T X).
 *
 * dh       : dh[M][F], leading dimension ld_dh, dtype x_dtype.
 * gu       : gu[M][2F] as written by fp8_gemm_gated, leading dimension ld_gu,
 *            dtype x_dtype.
 * mode     : FP8Q_SCALE_MAXABS or FP8Q_SCALE_POW2 (both tilings).
 * q        : 1x128 codes q[Mp][2F], leading dimension ld_q (bytes), with
 *            Mp = M rounded up to a multiple of 128.
 * scales   : their scales [2F/128][Mp], packed.
 * q_t      : 128x1 codes, transposed: q_t[2F][Mp], leading dimension ld_qt (bytes).
 * scales_t : their scales [Mp/128][2F], packed.
 *            The four are the operands of fp8_gemm_blockscaled DGRAD and WGRAD
 *            over Mp rows: rows M..Mp-1 of D are zeros.
 * dgu      : optional (NULL to skip): D itself, dgu[M][2F], leading dimension
 *            ld_dgu, dtype x_dtype, rounded once from FP32.
 * Requires F a multiple of 128.  M == 0 or F == 0 is a no-op.
 */
int fp8_gated_backward(int act, int64_t M, int64_t F,
                       const void* dh, int64_t ld_dh, const void* gu, int64_t ld_gu, int x_dtype,
                       int mode,
                       uint8_t* q, int64_t ld_q, float* scales,
                       uint8_t* q_t, int64_t ld_qt, float* scales_t,
                       void* dgu, int64_t ld_dgu,
                       void* stream);

/*
 * int8_quant_rows -- symmetric 8-bit codes with one scale for each row: a token
 * of an activation, an output channel of a weight stored [out][in].
 *   a = max(max_k |x[r][k]|, 127 * 2^-126)
 *   s = fl32(a * fl32(1/127)), inv = fl32(127 * fl32(1/a))  (IEEE operations)
 *   q = round-to-nearest-even(fl32(x * inv)), within [-127, 127]
 * The stored scale is the dequantization multiplier: x ~= s * q.
 *
 * x        : X[rows][cols], leading dimension ld_x, dtype x_dtype; any cols.
 * q        : codes [rows][cols], leading dimension ld_q (bytes); bytes beyond
 *            a row's cols are left as they are.
 * scales   : [rows].
 * rows == 0 is a no-op; cols == 0 writes the scale of a zero row.
 */
int int8_quant_rows(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                    int8_t* q, int64_t ld_q, float* scales,
                    void* stream);

/*
 * int8_gemm -- C[m][n] = a_scales[m] * b_scales[n] * sum_k A[m][k] B[n][k] (+ bias[n]).
 * The sum is exact (32-bit integers); the scales' product is formed in FP32
 * and multiplied in, the bias added, and the result rounded to C's dtype.
 *
 * a        : A[M][K] 8-bit integers, leading dimension lda (bytes).
 * a_scales : [M].
 * b        : B[N][K] 8-bit integers, leading dimension ldb (bytes).
 * b_scales : [N].
 * bias     : optional (NULL to skip): FP32 [N].
 * c        : C[M][N], leading dimension ldc, dtype c_dtype (FP8Q_BF16 or FP8Q_F32).
 * Any M, N and K from one token on.  Rows of A and B are read in whole
 * 16-byte chunks: the bytes from K up to the next multiple of 16 must be
 * readable in every row, the last one included, and the bytes between one row
 * and the next may be read; their values do not matter.
 * Every code from -128 to 127 is allowed.  K of at most 131,056 (beyond it the
 * 32-bit sum could overflow), lda, ldb of at most 4,194,176 bytes and at most
 * 2^31-1 tiles of 16x16 in C; otherwise FP8Q_ERR_UNSUPPORTED.  M == 0 or
 * N == 0 is a no-op; K == 0 writes the bias or zeros.
 */
int int8_gemm(int64_t M, int64_t N, int64_t K,
              const int8_t* a, int64_t lda, const float* a_scales,
              const int8_t* b, int64_t ldb, const float* b_scales,
              const float* bias,
              void* c, int c_dtype, int64_t ldc,
              void* stream);

/*
 * int8_gemm_gated -- fp8_gemm_gated's forward pass from 8-bit integers:
 *   g = int8_gemm(A, B[0:F]),  u = int8_gemm(A, B[F:2F])  (FP32, not rounded)
 *   h[m][f] = act(g[m][f]) * u[m][f]
 *
 * b        : B[2F][K], gate rows, then up rows; b_scales [2F].
 * h        : h[M][F], leading dimension ldh, dtype out_dtype.
 * Sizes, reads and limits as for int8_gemm, with any F.
 */
int int8_gemm_gated(int act, int64_t M, int64_t F, int64_t K,
                    const int8_t* a, int64_t lda, const float* a_scales,
                    const int8_t* b, int64_t ldb, const float* b_scales,
                    void* h, int out_dtype, int64_t ldh,
                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_FFN_H */
