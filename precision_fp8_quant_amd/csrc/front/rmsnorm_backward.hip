// Gradient of the root-mean-square norm.
//
//   xhat = h rstd,  g = dy w,  dx = rstd (g - xhat sum(g xhat) / D) + dh
//   dw[d] = sum_m dy[m][d] xhat[m][d]
// One pass over dy, h and dh: a row is held in registers between its sum and
// dx, by TPR threads of R runs of 8 elements (run i of thread t: columns
// 8 (i TPR + t)), and each thread keeps the sums of dw of its own columns over
// all rows of its workgroup.  The workgroups' sums (in the workspace, one row
// each) are added by a second kernel, in a fixed order: no atomics.
// Bound by memory: 8192x7168 BF16 with dh 83.6 us, 5.6 TB/s (a large copy: 5.1), and
// with the sums 86.3 among calls like it; each alone under a profiler 85.2 and 5.0,
// with the start and the end of a launch.  The registers of the sums decide the shape:
// 1024 threads of one run 91 us, 512 of two 93, 256 of four (one wave per SIMD) 107
// with 256 workgroups, both kernels alone; 512 workgroups 93, 2048, with 59 MB of
// sums, 109.
#include "front_launch.h"
#include "lanes.h"
#include "row_io.h"

namespace fp8q {
namespace {

// ONCE: dy, h and dh past the caches.
template <typename T, typename W, int TPR, int R, int NT, bool ONCE>
__global__ __launch_bounds__(NT) void rmsnorm_backward_kernel(NormBwdArgs p) {
  constexpr int RPB = NT / TPR;                    // rows at a time
  // With four runs the registers hold no more than dy and h: the sums of dw are in LDS, each thread's its own.  In FP32
  // they hold dy alone, and h is read again from the caches.  (2048x32768 with dh, us: BF16 114, with the sums in
  // registers, which spill, 194; FP32 343, with h in registers 390, the sums too 566.  With an FP32 weight the BF16 form
  // still spills 6 registers, 138; FP32 30.  With two runs FP32 spills 4 with a BF16 weight alone: 4096x16384 225, with an
  // FP32 one 213.)
  constexpr bool LATE = R > 2;
  constexpr bool AGAIN = LATE && sizeof(T) == 4;
  __shared__ v4f far[LATE ? 2 * R : 1][LATE ? TPR : 1];
  __shared__ float part[2][NT / 64];
  const int t = threadIdx.x & (TPR - 1);
  const T* __restrict__ dy = static_cast<const T*>(p.dy);
  const T* __restrict__ h = static_cast<const T*>(p.h);
  const T* __restrict__ dh = static_cast<const T*>(p.dh);
  T* __restrict__ dx = static_cast<T*>(p.dx);
  const W* __restrict__ weight = static_cast<const W*>(p.weight);
  const float inv_d = 1.0f / float(p.D);
  Row8<W> wr[R];
  float acc[LATE ? 1 : R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if constexpr (LATE) {
      far[2 * i][t] = far[2 * i + 1][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
      load_raw(wr[i], weight, (i * TPR + t) * 8, int(p.D));
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    }
  }
  int odd = 0;
  // the last rows' threads stay for the barriers (TPR > 64) and lane exchanges of the others
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < p.M; row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + threadIdx.x / TPR;
    const int D = row < p.M ? int(p.D) : 0;
    Row8<T> yr[R], hr[AGAIN ? 1 : R], er[R];
#pragma unroll
    for (int i = 0; i < R; ++i) load_raw<ONCE>(yr[i], dy + row * p.ld_dy, (i * TPR + t) * 8, D);
    if constexpr (!AGAIN) {
#pragma unroll
      for (int i = 0; i < R; ++i) load_raw<ONCE>(hr[i], h + row * p.ld_h, (i * TPR + t) * 8, D);
    }
    if (!LATE && dh) {
#pragma unroll
      for (int i = 0; i < R; ++i) load_raw<ONCE>(er[i], dh + row * p.ld_dh, (i * TPR + t) * 8, D);
    }
    const float rs = row < p.M ? p.rstd[row] : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int col = (i * TPR + t) * 8;
      if constexpr (LATE) load_raw(wr[i], weight, col, D);
      Row8<T>& hi = hr[AGAIN ? 0 : i];
      if constexpr (AGAIN) load_raw(hi, h + row * p.ld_h, col, D);
      trim(yr[i], col, D);
      trim(hi, col, D);
      trim(wr[i], col, int(p.D));
      float z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[j] = yr[i].get(j) * (hi.get(j) * rs);
        if constexpr (!LATE) acc[i][j] += z[j];
        sum = __builtin_fmaf(z[j], wr[i].get(j), sum);
      }
      if constexpr (LATE) {
        far[2 * i][t] += v4f{z[0], z[1], z[2], z[3]};
        far[2 * i + 1][t] += v4f{z[4], z[5], z[6], z[7]};
      }
      if constexpr (LATE) asm volatile("" ::: "memory");
    }
    const float c = row_sum<TPR>(sum, part[odd]) * inv_d;
    odd ^= 1;                                      // the next row's sums go to the other half: one barrier a row
#pragma unroll
    for (int i = 0; i < R; ++i) {
      yr[i].opaque();                              // unpacked again rather than held unpacked
      Row8<T>& hi = hr[AGAIN ? 0 : i];
      if constexpr (AGAIN) load_raw(hi, h + row * p.ld_h, (i * TPR + t) * 8, D);
      else hi.opaque();
      if constexpr (LATE) {
        load_raw(wr[i], weight, (i * TPR + t) * 8, D);
        if (dh) load_raw<ONCE>(er[i], dh + row * p.ld_dh, (i * TPR + t) * 8, D);
      }
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = rs * __builtin_fmaf(-(hi.get(j) * rs), c, yr[i].get(j) * wr[i].get(j));
        if (dh) v[j] += er[i].get(j);
      }
      store_raw(dx + row * p.ld_dx, (i * TPR + t) * 8, D, v);
      if constexpr (LATE) asm volatile("" ::: "memory");
    }
  }
  const int64_t dp = (p.D + 7) / 8 * 8;
  float* out = p.part + int64_t(blockIdx.x) * dp;
  if constexpr (RPB > 1) {                         // the rows of the workgroup meet in LDS
    __shared__ float sums[RPB][R * TPR * 8];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[threadIdx.x / TPR][(i * TPR + t) * 8 + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < dp; c += NT) {
      float s = sums[0][c];
#pragma unroll
      for (int k = 1; k < RPB; ++k) s += sums[k][c];
      out[c] = s;
    }
  } else if constexpr (LATE) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if ((i * TPR + t) * 8 < dp) {
        reinterpret_cast<v4f*>(out)[(i * TPR + t) * 2] = far[2 * i][t];
        reinterpret_cast<v4f*>(out)[(i * TPR + t) * 2 + 1] = far[2 * i + 1][t];
      }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if ((i * TPR + t) * 8 < dp) store8(out + (i * TPR + t) * 8, acc[i]);
  }
}

// dw[c] (+)= sum over the parts, 64 columns a workgroup, 16 waves that take the
// parts in turn (389 parts of 1999 columns: 3.1 us; 3.9 with 16 columns and four
// times the workgroups).
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ part, int64_t parts, int64_t ld,
                                                           int64_t cols, float* __restrict__ dw, bool accumulate) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t k = wave; k < parts; k += 16) s += part[k * ld + c];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += sums[w][lane];
    dw[c] = accumulate ? dw[c] + s : s;
  }
}

template <typename T, typename W, int TPR, int R, int NT>
void launch_rows(const NormBwdArgs& p, int64_t parts, hipStream_t st) {
  const dim3 grid{unsigned(parts)};
  if (p.once) hipLaunchKernelGGL((rmsnorm_backward_kernel<T, W, TPR, R, NT, true>), grid, dim3(NT), 0, st, p);
  else hipLaunchKernelGGL((rmsnorm_backward_kernel<T, W, TPR, R, NT, false>), grid, dim3(NT), 0, st, p);
}

template <typename T, typename W>
hipError_t launch(const NormBwdArgs& p, hipStream_t st) {
  int64_t parts = norm_bwd_parts(p.M, p.D);        // which counts on the rows of a workgroup here
  // BF16 rows of 1025 to 2048 channels, more than 512 of them: four at a time, in a quarter of the workgroups (with dh,
  // us in a graph, four / one: 1511x2048 9.7 / 11.4, 8192x2048 25.6 / 27.5, 32768x1536 78 / 93; 128x2048 5.7 / 5.2;
  // FP32, which has one everywhere, 1511x2048 13.3 / 14.5, 8192x2048 55.9 / 52.7, 32768x2048 198 / 188).
  const bool four = sizeof(T) == 2 && p.D > 1024 && p.D <= 2048 && p.M > 512;
  if (four) parts = p.M < 1024 ? (p.M + 3) / 4 : 256;   // never more than norm_bwd_parts says
  if (parts > 0) {
    if (four) {
      if constexpr (sizeof(T) == 2) launch_rows<T, W, 256, 1, 1024>(p, parts, st);
    } else if (p.D <= 128) launch_rows<T, W, 16, 1, 256>(p, parts, st);
    else if (p.D <= 256) launch_rows<T, W, 16, 2, 256>(p, parts, st);
    else if (p.D <= 512) launch_rows<T, W, 64, 1, 256>(p, parts, st);
    else if (p.D <= 1024) launch_rows<T, W, 64, 2, 256>(p, parts, st);
    else if (p.D <= 2048) launch_rows<T, W, 256, 1, 256>(p, parts, st);
    else if (p.D <= 4096) launch_rows<T, W, 512, 1, 512>(p, parts, st);
    else if (p.D <= 8192) launch_rows<T, W, 1024, 1, 1024>(p, parts, st);
    else if (p.D <= 16384) launch_rows<T, W, 1024, 2, 1024>(p, parts, st);
    else launch_rows<T, W, 1024, 4, 1024>(p, parts, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (parts == 0 && p.accumulate) return hipSuccess;
  hipLaunchKernelGGL(column_sums_kernel, dim3(unsigned((p.D + 63) / 64)), dim3(1024), 0, st, p.part, parts, (p.D + 7) / 8 * 8,
                     p.D, p.dw, p.accumulate);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_backward(const NormBwdArgs& p, bool x_bf16, bool w_bf16, hipStream_t st) {
  if (x_bf16) return w_bf16 ? launch<uint16_t, uint16_t>(p, st) : launch<uint16_t, float>(p, st);
  return w_bf16 ? launch<float, uint16_t>(p, st) : launch<float, float>(p, st);
}

}  // namespace fp8q
