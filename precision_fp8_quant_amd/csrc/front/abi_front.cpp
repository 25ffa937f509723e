// C ABI of the operators in front of the projections (include/fp8q_front.h):
// argument validation, then dispatch to the HIP launchers.  Every check runs on
// the host before anything is enqueued; the first violation returns its status
// and nothing is launched.
#include "../../../include/fp8q_front.h"
#include "../abi_check.hpp"
#include "front_launch.h"

#include <stdint.h>

namespace {

bool flag_ok(int v) { return v == 0 || v == 1; }
bool ld_ok(int64_t ld, int64_t es) { return ld % (16 / es) == 0; }

// A packed array of n elements.
Range packed(const void* p, int64_t n, int64_t es) { return span(p, p ? 1 : 0, n, n, es); }
Range matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  return span(p, p ? rows : 0, cols, ld, es);
}

template <int NO, int NI>
int check_ranges(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (const Range& r : outs)
    if (!r.ok) return FP8Q_ERR_SHAPE;
  for (const Range& r : ins)
    if (!r.ok) return FP8Q_ERR_SHAPE;
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i], ins[j])) return FP8Q_ERR_ALIAS;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return FP8Q_ERR_ALIAS;
  }
  return FP8Q_OK;
}

// What both norms ask of their common arguments (M > 0).
int check_norm(const fp8q::NormArgs& p, int64_t xs) {
  const bool cols = p.D > 0;
  if ((cols && (!p.x || !p.weight || !p.q || (p.r && !p.h))) || !p.scales) return FP8Q_ERR_NULL;
  if (cols && p.h && !p.r) return FP8Q_ERR_ARG;
  if (cols && (p.ld_x < p.D || (p.r && p.ld_r < p.D) || (p.h && p.ld_h < p.D) || (p.y && p.ld_y < p.D) || p.ld_q < p.D))
    return FP8Q_ERR_SHAPE;
  if (!aligned16(p.scales) || (p.rstd && !aligned16(p.rstd))) return FP8Q_ERR_ALIGN;
  if (cols && (!aligned16(p.x) || !aligned16(p.weight) || !aligned16(p.q) || !ld_ok(p.ld_x, xs) || p.ld_q % 16 ||
               (p.r && (!aligned16(p.r) || !ld_ok(p.ld_r, xs))) || (p.h && (!aligned16(p.h) || !ld_ok(p.ld_h, xs))) ||
               (p.y && (!aligned16(p.y) || !ld_ok(p.ld_y, xs)))))
    return FP8Q_ERR_ALIGN;
  if (p.D > fp8q::kMaxNormD) return FP8Q_ERR_UNSUPPORTED;
  return FP8Q_OK;
}

// Whether n inputs of M x D are more than the caches are good for.  D is at most
// kMaxNormD where it matters.
bool read_once(int64_t M, int64_t D, int64_t es, int64_t n) {
  return D > 0 && M > fp8q::kReadOnceBytes / (es * n) / D;
}

bool eps_ok(float eps) { return eps > 0.0f && eps <= 3.4028234664e38f; }   // false for NaN

bool route_sizes_ok(int64_t T, int64_t E, int64_t k, int64_t most) {
  return E >= 1 && E <= fp8q::kMaxExperts && k >= 1 && k <= fp8q::kMaxChosen && T <= (most - 1) / k;
}

}  // namespace

extern "C" {

int fp8_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int x_dtype, int64_t M, int64_t D,
                const void* weight, int w_dtype, float eps, int mode, void* h, int64_t ld_h, float* rstd, void* y,
                int64_t ld_y, uint8_t* q, int64_t ld_q, float* scales, uint8_t* q_t, int64_t ld_qt, float* scales_t,
                void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !eps_ok(eps)) return FP8Q_ERR_ARG;
  if (mode != FP8Q_SCALE_MAXABS && mode != FP8Q_SCALE_POW2) return FP8Q_ERR_ARG;
  if (M < 0 || D < 0) return FP8Q_ERR_SHAPE;
  if (M == 0 || D == 0) return FP8Q_OK;
  const int64_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  const fp8q::NormArgs p{x, ld_x, residual, ld_r, M, D, weight, eps, h, ld_h, rstd, y, ld_y, q, ld_q, scales, q_t, ld_qt,
                         scales_t, read_once(M, D, xs, residual ? 2 : 1)};
  if (!q_t != !scales_t) return FP8Q_ERR_NULL;
  if (q_t && !rstd) return FP8Q_ERR_NULL;
  const int bad = check_norm(p, xs);
  if (bad != FP8Q_OK) return bad;
  int64_t mp = M, n1 = 0, n2 = 0;
  if (q_t) {
    if (__builtin_add_overflow(M, 127, &mp)) return FP8Q_ERR_SHAPE;
    mp -= mp % 128;
    if (ld_qt < mp) return FP8Q_ERR_SHAPE;
    if (!aligned16(q_t) || !aligned16(scales_t) || ld_qt % 16) return FP8Q_ERR_ALIGN;
  }
  if (D % 128) return FP8Q_ERR_UNSUPPORTED;
  if (!mul_ok(D / 128, mp, &n1) || !mul_ok(mp / 128, D, &n2)) return FP8Q_ERR_SHAPE;
  const Range outs[7] = {matrix(h, M, D, ld_h, xs), packed(rstd, M, 4), matrix(y, M, D, ld_y, xs), matrix(q, mp, D, ld_q, 1),
                         packed(scales, n1, 4), matrix(q_t, D, mp, ld_qt, 1), packed(scales_t, n2, 4)};
  const Range ins[3] = {matrix(x, M, D, ld_x, xs), matrix(residual, M, D, ld_r, xs), packed(weight, D, ws)};
  const int clash = check_ranges(outs, ins);
  if (clash != FP8Q_OK) return clash;
  return from_hip(fp8q::launch_fp8_rmsnorm(p, x_dtype == FP8Q_BF16, w_dtype == FP8Q_BF16, mode,
                                           reinterpret_cast<hipStream_t>(stream)));
}

int int8_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int x_dtype, int64_t M, int64_t D,
                 const void* weight, int w_dtype, float eps, void* h, int64_t ld_h, float* rstd, void* y, int64_t ld_y,
                 int8_t* q, int64_t ld_q, float* scales, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !eps_ok(eps)) return FP8Q_ERR_ARG;
  if (M < 0 || D < 0) return FP8Q_ERR_SHAPE;
  if (M == 0) return FP8Q_OK;
  const int64_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  const fp8q::NormArgs p{x, ld_x, residual, ld_r, M, D, weight, eps, h, ld_h, rstd, y, ld_y,
                         reinterpret_cast<uint8_t*>(q), ld_q, scales, nullptr, 0, nullptr,
                         read_once(M, D, xs, residual ? 2 : 1)};
  const int bad = check_norm(p, xs);
  if (bad != FP8Q_OK) return bad;
  const Range outs[5] = {matrix(h, M, D, ld_h, xs), packed(rstd, M, 4), matrix(y, M, D, ld_y, xs), matrix(q, M, D, ld_q, 1),
                         packed(scales, M, 4)};
  const Range ins[3] = {matrix(x, M, D, ld_x, xs), matrix(residual, M, D, ld_r, xs), packed(weight, D, ws)};
  const int clash = check_ranges(outs, ins);
  if (clash != FP8Q_OK) return clash;
  return from_hip(fp8q::launch_int8_rmsnorm(p, x_dtype == FP8Q_BF16, w_dtype == FP8Q_BF16,
                                            reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8q_rmsnorm_backward_workspace(int64_t M, int64_t D) {
  return M < 0 || D < 0 || D > fp8q::kMaxNormD ? -1 : fp8q::norm_bwd_workspace(M, D);
}

int rmsnorm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, int x_dtype, int64_t M, int64_t D,
                     const void* weight, int w_dtype, const float* rstd, const void* dh, int64_t ld_dh, void* dx,
                     int64_t ld_dx, float* dw, int accumulate, void* workspace, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_dtype) || !flag_ok(accumulate)) return FP8Q_ERR_ARG;
  if (M < 0 || D < 0) return FP8Q_ERR_SHAPE;
  if (D == 0) return FP8Q_OK;
  const bool rows = M > 0, wide = D > fp8q::kMaxNormD;     // wide: no workspace has a size
  if (!dw || (rows && (!dy || !h || !weight || !rstd || !dx || (!workspace && !wide)))) return FP8Q_ERR_NULL;
  if (rows && (ld_dy < D || ld_h < D || ld_dx < D || (dh && ld_dh < D))) return FP8Q_ERR_SHAPE;
  const int64_t xs = dtype_size(x_dtype), ws = dtype_size(w_dtype);
  if (!aligned16(dw) || (rows && (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(rstd) ||
                                  !aligned16(dx) || !aligned16(workspace) || !ld_ok(ld_dy, xs) || !ld_ok(ld_h, xs) ||
                                  !ld_ok(ld_dx, xs) || (dh && (!aligned16(dh) || !ld_ok(ld_dh, xs))))))
    return FP8Q_ERR_ALIGN;
  if (wide) return FP8Q_ERR_UNSUPPORTED;
  const int64_t m1 = rows ? 1 : 0;
  const Range outs[3] = {matrix(dx, M, D, ld_dx, xs), packed(dw, D, 4),
                         packed(workspace, m1 * fp8q::norm_bwd_workspace(M, D), 1)};
  const Range ins[5] = {matrix(dy, M, D, ld_dy, xs), matrix(h, M, D, ld_h, xs), packed(weight, m1 * D, ws),
                        packed(rstd, M, 4), matrix(dh, M, D, ld_dh, xs)};
  const int clash = check_ranges(outs, ins);
  if (clash != FP8Q_OK) return clash;
  const fp8q::NormBwdArgs p{dy, ld_dy, h, ld_h, M, D, weight, rstd, dh, ld_dh, dx, ld_dx, dw, accumulate == 1,
                            static_cast<float*>(workspace), read_once(M, D, xs, dh ? 3 : 2)};
  return from_hip(fp8q::launch_rmsnorm_backward(p, x_dtype == FP8Q_BF16, w_dtype == FP8Q_BF16,
                                                reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8q_moe_route_workspace(int64_t T, int64_t E) {
  if (T < 0 || !route_sizes_ok(T, E, 1, int64_t(1) << 31)) return -1;
  return fp8q::route_workspace(T, E);
}

int moe_route(const void* logits, int64_t ld_z, int z_dtype, int64_t T, int64_t E, int64_t k, const uint8_t* valid,
              int renormalize, float* weights, int32_t* experts, int32_t* counts, float* loss, float* slope,
              void* workspace, void* stream) {
  if (!dtype_ok(z_dtype) || !flag_ok(renormalize)) return FP8Q_ERR_ARG;
  if (T < 0 || E < 0 || k < 0 || k > E) return FP8Q_ERR_SHAPE;
  if (!route_sizes_ok(T, E, k, int64_t(1) << 31)) return FP8Q_ERR_UNSUPPORTED;
  const int64_t bytes = fp8q::route_workspace(T, E), zs = dtype_size(z_dtype);
  if (!counts || !loss || !slope || (T > 0 && (!logits || !weights || !experts)) || (bytes > 0 && !workspace))
    return FP8Q_ERR_NULL;
  if (T > 0 && ld_z < E) return FP8Q_ERR_SHAPE;
  if (!aligned16(counts) || !aligned16(loss) || !aligned16(slope) || (bytes > 0 && !aligned16(workspace)) ||
      (valid && !aligned16(valid)) ||
      (T > 0 && (!aligned16(logits) || !aligned16(weights) || !aligned16(experts) || !ld_ok(ld_z, zs))))
    return FP8Q_ERR_ALIGN;
  const Range outs[6] = {packed(weights, T * k, 4), packed(experts, T * k, 4), packed(counts, E, 4), packed(loss, 1, 4),
                         packed(slope, E, 4), packed(workspace, bytes, 1)};
  const Range ins[2] = {matrix(logits, T, E, ld_z, zs), packed(valid, T, 1)};
  const int clash = check_ranges(outs, ins);
  if (clash != FP8Q_OK) return clash;
  const int64_t parts = fp8q::route_parts(T, E);
  float* pp = static_cast<float*>(workspace);
  int32_t* pc = bytes > 0 ? reinterpret_cast<int32_t*>(pp + parts * E) : nullptr;
  int32_t* pn = bytes > 0 ? pc + parts * E : nullptr;
  float* pl = bytes > 0 ? reinterpret_cast<float*>(pn + (parts + 3) / 4 * 4) : nullptr;
  const fp8q::RouteArgs p{logits, ld_z, T, E, k, valid, renormalize == 1, weights, experts, counts, loss, slope, pp, pc, pn,
                          pl};
  return from_hip(fp8q::launch_moe_route(p, z_dtype == FP8Q_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int moe_route_backward(const void* logits, int64_t ld_z, int z_dtype, int64_t T, int64_t E, int64_t k,
                       const int32_t* experts, const float* slope, const float* dweights, const float* dloss,
                       int renormalize, void* dlogits, int64_t ld_dz, void* stream) {
  if (!dtype_ok(z_dtype) || !flag_ok(renormalize)) return FP8Q_ERR_ARG;
  if (T < 0 || E < 0 || k < 0 || k > E) return FP8Q_ERR_SHAPE;
  if (!route_sizes_ok(T, E, k, int64_t(1) << 31)) return FP8Q_ERR_UNSUPPORTED;
  if (T == 0) return FP8Q_OK;
  if (!logits || !experts || !dlogits || (dloss && !slope)) return FP8Q_ERR_NULL;
  if (ld_z < E || ld_dz < E) return FP8Q_ERR_SHAPE;
  const int64_t zs = dtype_size(z_dtype);
  if (!aligned16(logits) || !aligned16(experts) || !aligned16(dlogits) || !ld_ok(ld_z, zs) || !ld_ok(ld_dz, zs) ||
      (slope && !aligned16(slope)) || (dweights && !aligned16(dweights)) || (dloss && !aligned16(dloss)))
    return FP8Q_ERR_ALIGN;
  const Range outs[1] = {matrix(dlogits, T, E, ld_dz, zs)};
  const Range ins[5] = {matrix(logits, T, E, ld_z, zs), packed(experts, T * k, 4), packed(slope, E, 4),
                        packed(dweights, T * k, 4), packed(dloss, 1, 4)};
  const int clash = check_ranges(outs, ins);
  if (clash != FP8Q_OK) return clash;
  const fp8q::RouteBwdArgs p{logits, ld_z, T, E, k, experts, slope, dweights, dloss, renormalize == 1, dlogits, ld_dz};
  return from_hip(fp8q::launch_moe_route_backward(p, z_dtype == FP8Q_BF16, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8q_moe_max_rows(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || !route_sizes_ok(T, E, k, int64_t(1) << 30)) return -1;
  return fp8q::dispatch_max_rows(T * k, E);
}

int64_t fp8q_moe_dispatch_workspace(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || !route_sizes_ok(T, E, k, int64_t(1) << 30)) return -1;
  return fp8q::dispatch_workspace(T * k, E);
}

int fp8_moe_dispatch(const int32_t* experts, int64_t T, int64_t k, int64_t E, const uint8_t* q, int64_t ld_q,
                     const float* scales, int64_t D, int64_t M_total, uint8_t* a, int64_t ld_a, float* a_scales,
                     int32_t* group_of_mtile, int32_t* row_of_slot, int32_t* token_of_row, void* workspace,
                     void* stream) {
  if (T < 0 || k < 0 || E < 0 || D < 0 || M_total < 0) return FP8Q_ERR_SHAPE;
  if (!route_sizes_ok(T, E, k, int64_t(1) << 30)) return FP8Q_ERR_UNSUPPORTED;
  if (M_total % 128 || M_total < fp8q::dispatch_max_rows(T * k, E)) return FP8Q_ERR_SHAPE;
  const int64_t bytes = fp8q::dispatch_workspace(T * k, E);
  const bool moves = T > 0 && D > 0;
  if ((T > 0 && (!experts || !row_of_slot)) || (M_total > 0 && (!group_of_mtile || !token_of_row)) ||
      (moves && (!q || !scales || !a || !a_scales)) || (bytes > 0 && !workspace))
    return FP8Q_ERR_NULL;
  if (moves && (ld_q < D || ld_a < D)) return FP8Q_ERR_SHAPE;
  if ((T > 0 && (!aligned16(experts) || !aligned16(row_of_slot))) ||
      (M_total > 0 && (!aligned16(group_of_mtile) || !aligned16(token_of_row))) ||
      (moves && (!aligned16(q) || !aligned16(scales) || !aligned16(a) || !aligned16(a_scales) || ld_q % 16 || ld_a % 16)) ||
      (bytes > 0 && !aligned16(workspace)))
    return FP8Q_ERR_ALIGN;
  if (D % 128 || M_total > (int64_t(1) << 31) - 128) return FP8Q_ERR_UNSUPPORTED;
  int64_t ns = 0, na = 0;
  if (!mul_ok(D / 128, T, &ns) || !mul_ok(D / 128, M_total, &na)) return FP8Q_ERR_SHAPE;
  const Range outs[6] = {matrix(a, moves ? M_total : 0, D, ld_a, 1), packed(a_scales, moves ? na : 0, 4),
                         packed(group_of_mtile, M_total / 128, 4), packed(row_of_slot, T * k, 4),
                         packed(token_of_row, M_total, 4), packed(workspace, bytes, 1)};
  const Range ins[3] = {packed(experts, T * k, 4), matrix(q, moves ? T : 0, D, ld_q, 1), packed(scales, moves ? ns : 0, 4)};
  const int clash = check_ranges(outs, ins);
  if (clash != FP8Q_OK) return clash;
  if (M_total == 0) return FP8Q_OK;               // no slots and no tiles
  const fp8q::DispatchArgs p{experts, T, k, E, q, ld_q, scales, D, M_total, a, ld_a, a_scales, group_of_mtile, row_of_slot,
                             token_of_row, static_cast<int32_t*>(workspace)};
  return from_hip(fp8q::launch_moe_dispatch(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
