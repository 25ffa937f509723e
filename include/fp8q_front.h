/*
 * fp8q -- operators in front of the projections for AMD Instinct MI355X
 * (gfx950).  C ABI, exported by the same library as include/fp8q.h.
 *
 * A root-mean-square norm that adds the residual and hands its result on in
 * the 8-bit forms that the products take (fp8_rmsnorm, int8_rmsnorm), its
 * gradient (rmsnorm_backward); the choice of experts with the tokens of each
 * expert and the loss that balances them (moe_route, moe_route_backward); and
 * the rows of codes in the order of their experts, as
 * fp8_gemm_blockscaled_grouped takes them (fp8_moe_dispatch).
 *
 * Every convention of fp8q.h holds here: device pointers owned by the caller,
 * no allocation, no state, no synchronisation, all work on `stream`, plain int
 * status codes and enum values, arguments validated before anything is
 * launched, row-major matrices with leading dimensions in elements, 16-byte
 * aligned pointers and leading dimensions of a multiple of 16 bytes, finite
 * inputs (but for the logits of moe_route, see there), outputs that overlap
 * neither inputs nor each other.  Rows of inputs are read in whole 16-byte
 * chunks: the bytes from their last column up to the next multiple of 16 may be
 * read, and their values do not matter.  Bytes of an output's row beyond its
 * columns are left as they are.
 *
 * A workspace is scratch memory of the caller's, 16-byte aligned, of the bytes
 * that the operator's own *_workspace function says (0: none, may be NULL;
 * -1: no such sizes).  What it holds before a call does not matter; two calls
 * that may run at the same time need one each.
 *
 * Sums over rows and columns, probabilities and norms are FP32.  Results do
 * not depend on timing: sums are taken in a fixed order.
 */
#ifndef FP8Q_FRONT_H
#define FP8Q_FRONT_H

#include "fp8q.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8_rmsnorm -- norm of x (+ residual), quantized to FP8:
 *   h = x + residual  (FP32, rounded to x_dtype: the stream that goes on), or h = x
 *   rstd = 1 / sqrt(mean_d h^2 + eps)
 *   y[m][d] = (h[m][d] rstd[m]) weight[d]
 * The norm is that of the rounded h, so that rmsnorm_backward differentiates
 * what was computed.  y is quantized from FP32 by the rule of fp8q.h.
 *
 * x, residual : X[M][D], leading dimensions ld_x, ld_r, dtype x_dtype;
 *            residual is optional (NULL to skip).
 * weight   : [D], dtype w_dtype.
 * eps      : > 0 and finite.
 * mode     : FP8Q_SCALE_MAXABS or FP8Q_SCALE_POW2 (both tilings).
 * h        : H[M][D], leading dimension ld_h, x_dtype; required with residual,
 *            NULL without.
 * rstd     : [M]; optional (NULL to skip), required with q_t.
 * y        : optional (NULL to skip): Y[M][D], leading dimension ld_y, x_dtype,
 *            rounded once from FP32.
 * q        : 1x128 codes q[Mq][D], leading dimension ld_q (bytes).  Mq is M; with
 *            q_t it is Mp, M rounded up to a multiple of 128, and the rows
 *            M..Mp-1 are those of zeros.
 * scales   : their scales [D/128][Mq], packed.
 * q_t, scales_t : optional (both NULL to skip): 128x1 codes, transposed,
 *            q_t[D][Mp], leading dimension ld_qt (bytes), and their scales
 *            [Mp/128][D], packed: the operand of fp8_gemm_blockscaled WGRAD.
 * Requires D a multiple of 128, at most 32768 (FP8Q_ERR_UNSUPPORTED).  The sum
 * of squares of a row of h, and y, must be finite in FP32.  M == 0 or D == 0 is
 * a no-op.
 */
int fp8_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int x_dtype,
                int64_t M, int64_t D,
                const void* weight, int w_dtype, float eps, int mode,
                void* h, int64_t ld_h, float* rstd, void* y, int64_t ld_y,
                uint8_t* q, int64_t ld_q, float* scales,
                uint8_t* q_t, int64_t ld_qt, float* scales_t,
                void* stream);

/*
 * int8_rmsnorm -- the same norm in 8-bit integers with one scale for each row,
 * by the rule of int8_quant_rows (fp8q_ffn.h) on the FP32 y.
 *
 * q        : codes q[M][D], leading dimension ld_q (bytes).
 * scales   : [M].
 * Any D up to 32768 (FP8Q_ERR_UNSUPPORTED beyond).  M == 0 is a no-op; D == 0
 * writes the scale of a zero row (and rstd of one, 1 / sqrt(eps)).
 */
int int8_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int x_dtype,
                 int64_t M, int64_t D,
                 const void* weight, int w_dtype, float eps,
                 void* h, int64_t ld_h, float* rstd, void* y, int64_t ld_y,
                 int8_t* q, int64_t ld_q, float* scales,
                 void* stream);

/*
 * rmsnorm_backward -- gradient of the norm's y with respect to its input and
 * its weight:
 *   xhat = h rstd,  g = dy weight
 *   dx = rstd (g - xhat mean_d(g xhat)) + dh,   dw[d] (+)= sum_m dy[m][d] xhat[m][d]
 * x and residual enter h as a sum: dx is the gradient of both.
 *
 * dy       : dY[M][D], leading dimension ld_dy, dtype x_dtype.
 * h, rstd  : what the forward pass normed (x where it had no residual) and its rstd.
 * dh       : optional (NULL to skip): dH[M][D], leading dimension ld_dh, x_dtype:
 *            the gradient that reaches h past the norm.
 * dx       : dX[M][D], leading dimension ld_dx, x_dtype, rounded once from FP32.
 * dw       : FP32 [D].  accumulate 0: written; 1: added to.
 * workspace: fp8q_rmsnorm_backward_workspace(M, D) bytes.
 * Any D up to 32768 (FP8Q_ERR_UNSUPPORTED beyond).  D == 0 is a no-op; M == 0
 * writes zeros to dw, or leaves it with accumulate.
 */
int rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, int x_dtype,
                     int64_t M, int64_t D,
                     const void* weight, int w_dtype, const float* rstd,
                     const void* dh, int64_t ld_dh,
                     void* dx, int64_t ld_dx, float* dw, int accumulate,
                     void* workspace, void* stream);
int64_t fp8q_rmsnorm_backward_workspace(int64_t M, int64_t D);

/*
 * moe_route -- the k experts of each token:
 *   p[t][e] = softmax_e(logits[t][e])
 *   experts[t] = the k experts of the largest logits, in descending order (the
 *                lower index first where they are equal)
 *   weights[t][j] = p[t][experts[t][j]], or that over the sum of the chosen ones
 *   counts[e] = how often e was chosen
 *   loss = E sum_e f_e P_e,  f_e = counts[e] / (k n),  P_e = 1/n sum_t p[t][e]
 * over the n tokens that count; 1 where all experts share evenly.  Its slope
 * by p[t][e] is the same for every token that counts: slope[e] =
 * E counts[e] / (k n^2), the counts being constants of the gradient.
 *
 * logits   : Z[T][E], leading dimension ld_z, dtype z_dtype.  Minus infinity
 *            takes an expert out of a token's choice: it has p = 0 and is never
 *            chosen.  A token with fewer than k others gets them alone, and
 *            expert -1 with weight 0 in the remaining places.
 * valid    : optional (NULL: all): uint8 [T]; 0 for a token that does not
 *            count, whose logits do not matter.  It, and a token whose logits
 *            are all minus infinity, has experts -1 and weights 0.
 * renormalize : 0 or 1.
 * weights  : FP32 [T][k], packed.   experts : int32 [T][k], packed.
 * counts   : int32 [E].   loss : FP32 [1].   slope : FP32 [E].  Zeros where no
 *            token counts.
 * workspace: fp8q_moe_route_workspace(T, E) bytes.
 * Requires 1 <= E <= 1024, 1 <= k <= min(E, 32) and T k < 2^31
 * (FP8Q_ERR_UNSUPPORTED).  NaN or plus infinity among the logits of a token
 * that counts gives unspecified weights, loss and slope; experts stay within
 * [-1, E).  T == 0 writes zeros to counts, loss and slope.
 */
int moe_route(const void* logits, int64_t ld_z, int z_dtype, int64_t T, int64_t E, int64_t k,
              const uint8_t* valid, int renormalize,
              float* weights, int32_t* experts, int32_t* counts, float* loss, float* slope,
              void* workspace, void* stream);
int64_t fp8q_moe_route_workspace(int64_t T, int64_t E);

/*
 * moe_route_backward -- gradient with respect to the logits:
 *   dp[t][e] = dloss slope[e] + sum over the j with experts[t][j] == e of dc[t][j]
 *   dlogits[t][e] = p[t][e] (dp[t][e] - sum_i p[t][i] dp[t][i])
 * dc is dweights, or its gradient through the renormalization,
 * (dweights[t][j] - sum_i dweights[t][i] weights[t][i]) / (sum of the chosen p).
 *
 * logits, experts, slope, renormalize : as in moe_route.
 * dweights : optional (NULL: zero): FP32 [T][k], packed.
 * dloss    : optional (NULL: zero): FP32 [1] on the device, the gradient that
 *            reaches the loss (the loss's coefficient included).
 * dlogits  : dZ[T][E], leading dimension ld_dz, z_dtype, rounded once from FP32.
 *            Zeros for tokens that do not count (experts[t][0] < 0), whose
 *            logits and dweights do not matter.
 * Other experts outside [0, E) contribute nothing.  Sizes as in moe_route; T == 0 is
 * a no-op.
 */
int moe_route_backward(const void* logits, int64_t ld_z, int z_dtype, int64_t T, int64_t E, int64_t k,
                       const int32_t* experts, const float* slope, const float* dweights, const float* dloss,
                       int renormalize,
                       void* dlogits, int64_t ld_dz,
                       void* stream);

/*
 * fp8_moe_dispatch -- rows of codes in the order of their experts, each
 * expert's rows padded to whole 128-row tiles: A, its scales and the tile map
 * of fp8_gemm_blockscaled_grouped.
 *   c_e rows for expert e, first row s_e = 128 sum_{i<e} ceil(c_i / 128)
 *   row_of_slot[t][j] = s_e + (slots of e before (t, j)),  e = experts[t][j]
 *
 * experts  : int32 [T][k], packed.  A slot whose expert is outside [0, E) gets
 *            no row, and row_of_slot -1.
 * q, scales: codes Q[T][D] (leading dimension ld_q, bytes) and 1x128 scales
 *            [D/128][T], packed (fp8_rmsnorm, fp8_quant_tile).
 * M_total  : rows of A: a multiple of 128 of at least fp8q_moe_max_rows(T, k, E).
 * a        : A[M_total][D], leading dimension ld_a (bytes).  Padding rows of a
 *            tile in use are zeros with the scale of zeros, 2^-126; rows and
 *            scales of tiles past the last one in use are left as they are.
 * a_scales : [D/128][M_total], packed.
 * group_of_mtile : int32 [M_total/128]; -1 for tiles that are not in use.
 * row_of_slot    : int32 [T][k], packed.
 * token_of_row   : int32 [M_total]; -1 for rows that hold no token.
 * workspace: fp8q_moe_dispatch_workspace(T, k, E) bytes.
 * Requires D a multiple of 128, 1 <= E <= 1024, 1 <= k <= 32, T k < 2^30 and
 * M_total < 2^31 (FP8Q_ERR_UNSUPPORTED).  T == 0 or D == 0 still writes the maps.
 */
int fp8_moe_dispatch(const int32_t* experts, int64_t T, int64_t k, int64_t E,
                     const uint8_t* q, int64_t ld_q, const float* scales, int64_t D,
                     int64_t M_total,
                     uint8_t* a, int64_t ld_a, float* a_scales,
                     int32_t* group_of_mtile, int32_t* row_of_slot, int32_t* token_of_row,
                     void* workspace, void* stream);
int64_t fp8q_moe_max_rows(int64_t T, int64_t k, int64_t E);
int64_t fp8q_moe_dispatch_workspace(int64_t T, int64_t k, int64_t E);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_FRONT_H */
