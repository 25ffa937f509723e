// Root-mean-square norm with the residual's addition, in 8 bits.
//
//   h = T(x + r),  rstd = 1 / sqrt(sum h^2 / D + eps),  y = (h rstd) w
// y leaves as FP8 codes in 1x128 tiles or as 8-bit integers with a scale for
// the row, both quantized from FP32.
//
// A streaming pass, bound by memory: the row is read once and held in registers
// between its sum of squares and its codes.  TPR threads share a row and hold R
// runs of 8 elements each, run i of thread t being columns 8 (i TPR + t): a DPP
// row of 16 lanes holds a 1x128 tile.  Measured (a large copy: 5.1 TB/s): 8192x7168
// BF16 with a residual and y 89 us, 5.9 TB/s; 1511x2048 FP32 with a residual and y
// 11.6 us; one token 4.0 us, a launch and two trips to memory.
#include "../fp8q_launch.h"
#include "front_launch.h"
#include "lanes.h"
#include "row_io.h"

namespace fp8q {
namespace {

enum { kOutFp8, kOutFp8Pow2, kOutInt8, kOutNone };

// A product of |y| <= a with inv <= (448 / a)(1 + 2^-24) rounds to at most the
// code of 448, so no clamp is needed before the conversion.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

__device__ __forceinline__ float max_abs8(const float (&v)[8]) {
  float m = __builtin_fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
  return m;
}

// ONCE: x and the residual past the caches.
template <typename T, typename W, int TPR, int R, int OUT, bool ONCE>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_kernel(NormArgs p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  // With four runs of 1024 threads the registers hold no weight before the sum (512x32768 FP32, us: 21.6, with it, which
  // spills, 30.2; with a residual 50 and 67).
  constexpr bool LATE = TPR * R > 2048;
  __shared__ float part[2][NT / 64];
  const int t = threadIdx.x & (TPR - 1);
  const T* __restrict__ x = static_cast<const T*>(p.x);
  const T* __restrict__ r = static_cast<const T*>(p.r);
  T* __restrict__ h = static_cast<T*>(p.h);
  T* __restrict__ y = static_cast<T*>(p.y);
  const W* __restrict__ weight = static_cast<const W*>(p.weight);
  const float inv_d = p.D > 0 ? 1.0f / float(p.D) : 0.0f;
  // the last rows' threads stay for the barriers (TPR > 64) and lane exchanges of the others
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < p.M; row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + threadIdx.x / TPR;
    const int D = row < p.M ? int(p.D) : 0;
    Row8<T> xr[R], rr[R];
    Row8<W> wr[R];
#pragma unroll
    for (int i = 0; i < R; ++i) load_raw<ONCE>(xr[i], x + row * p.ld_x, (i * TPR + t) * 8, D);
    if (r) {
#pragma unroll
      for (int i = 0; i < R; ++i) load_raw<ONCE>(rr[i], r + row * p.ld_r, (i * TPR + t) * 8, D);
    }
    if constexpr (OUT != kOutNone && !LATE) {
#pragma unroll
      for (int i = 0; i < R; ++i) load_raw(wr[i], weight, (i * TPR + t) * 8, D);
    }
    float v[R][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int col = (i * TPR + t) * 8;
      trim(xr[i], col, D);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = xr[i].get(j);
      if (r) {
        trim(rr[i], col, D);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += rr[i].get(j);
        store_raw(h + row * p.ld_h, col, D, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = held(v[i][j], T());
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(v[i][j], v[i][j], sum);
    }
    sum = row_sum<TPR>(sum, part[0]);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, inv_d, p.eps));
    if (p.rstd && t == 0 && row < p.M) p.rstd[row] = rstd;
    if constexpr (OUT != kOutNone) {
      float row_a = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int col = (i * TPR + t) * 8;
        if constexpr (LATE) load_raw(wr[i], weight, col, D);
        trim(wr[i], col, D);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * wr[i].get(j);
        if (y) store_raw(y + row * p.ld_y, col, D, v[i]);
        const float a = max_abs8(v[i]);
        if constexpr (OUT == kOutInt8) {
          row_a = __builtin_fmaxf(row_a, a);
        } else {
          constexpr int MODE = OUT == kOutFp8Pow2 ? kModePow2 : kModeMaxAbs;
          const ScalePair sp = scale_from_amax_bits<MODE>(row16_max_u32(__float_as_uint(a)));
          if (col < D) {
            *reinterpret_cast<uint2*>(p.q + row * p.ld_q + col) =
                uint2{quant4(v[i][0], v[i][1], v[i][2], v[i][3], sp.inv), quant4(v[i][4], v[i][5], v[i][6], v[i][7], sp.inv)};
            if ((t & 15) == 0) p.scales[int64_t(col >> 7) * p.M + row] = sp.s;
          }
        }
      }
      if constexpr (OUT == kOutInt8) {
        const float a = __builtin_fmaxf(row_max<TPR>(row_a, part[1]), __uint_as_float(kInt8FloorBits));
        const float inv = (1.0f / a) * 127.0f;
        if (t == 0 && row < p.M) p.scales[row] = a * (1.0f / 127.0f);
        int8_t* q = reinterpret_cast<int8_t*>(p.q) + row * p.ld_q;
#pragma unroll
        for (int i = 0; i < R; ++i) store_run(q, (i * TPR + t) * 8, D, v[i], inv);
      }
    }
    if constexpr (TPR > 64) __syncthreads();       // `part` is reused by the next row
  }
}

// ---------------------------------------------------------------------------
// Both FP8 tilings, from the stream h and its rstd that the kernel above left.
// One 512-thread workgroup per 128x128 block; thread t owns the 8 columns
// 8*(t%16)..+7 of the rows 4*(t/16)..+3, so a DPP row holds a 1x128 tile.
// Column maxima go over the thread's rows, the wave (permlane swaps) and the 8
// waves (LDS); transposed codes are staged in LDS and leave 32 bytes a thread.
// Rows past M are zeros.
// Bound by memory: 8192x7168 BF16 41 us, 5.9 TB/s, after 55 us (6.4 TB/s) of the
// kernel above with a residual.  It is a second kernel because a column's tile
// needs the rstd of 128 rows, more than a CU holds; its read of h is what the two
// passes pay for that, and comes out of the caches in part.
// ---------------------------------------------------------------------------
constexpr int kPitch = 132;    // bytes per LDS row of the transposed tile

template <typename T, typename W, int MODE>
__global__ __launch_bounds__(512) void rmsnorm_dual_kernel(NormArgs p) {
  __shared__ float col_part[8][128];
  __shared__ __attribute__((aligned(16))) float inv_col[128];
  __shared__ uint32_t tile[128 * kPitch / 4];
  const T* __restrict__ h = static_cast<const T*>(p.h);
  T* __restrict__ y = static_cast<T*>(p.y);
  const W* __restrict__ weight = static_cast<const W*>(p.weight);
  const float* __restrict__ rstd = p.rstd;
  const int t = threadIdx.x, c16 = t & 15, rq = t >> 4;
  const int64_t cblocks = p.D >> 7, rblocks = (p.M + 127) >> 7, mp = rblocks << 7;
  for (int64_t u = blockIdx.x; u < cblocks * rblocks; u += gridDim.x) {   // block-uniform: barriers stay matched
    // Four row blocks at a time, which extend the same 512 bytes of q_t.  Measured (8192x7168 BF16, inputs from memory, with
    // a residual / without, us a call that writes where the last one's dropped outputs were, and one whose last outputs are
    // still held): 92.4 / 67.3 and 103.7 / 69.4; row by row 93.3 / 68.5 and 103.9 / 70.6, column by column 92.9 / 71.5 and
    // 107.8 / 72.4; fours from the end, where h was written last, 92.7 / 68.1 and 106.6 / 73.0.
    const int64_t first = u / (4 * cblocks) * 4, left = rblocks - first, high = left < 4 ? left : 4, v4 = u % (4 * cblocks);
    const int64_t br = first + v4 % high, bc = v4 / high;
    const int64_t col = bc * 128 + c16 * 8, row0 = br * 128 + rq * 4;
    Row8<T> hr[4];
    Row8<W> wr;
    float rs[4], v[4][8];
    wr.load(weight + col);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rs[j] = 0.0f;
      if (row0 + j < p.M) {
        hr[j].load(h + (row0 + j) * p.ld_h + col);
        rs[j] = rstd[row0 + j];
      } else {
        hr[j].zero();
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = row0 + j < p.M ? hr[j].get(i) * rs[j] * wr.get(i) : 0.0f;   // no -0 past M
      if (y && row0 + j < p.M) store8(y + (row0 + j) * p.ld_y + col, v[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(v[0][i]), __builtin_fabsf(v[1][i])),
                                      __builtin_fmaxf(__builtin_fabsf(v[2][i]), __builtin_fabsf(v[3][i])));
      const uint32_t b = __float_as_uint(m);       // lanes l, l^16, l^32, l^48 hold the same column
      const auto a = __builtin_amdgcn_permlane32_swap(b, b, false, false);
      const uint32_t c = uint32_t(a[0]) > uint32_t(a[1]) ? uint32_t(a[0]) : uint32_t(a[1]);
      const auto d = __builtin_amdgcn_permlane16_swap(c, c, false, false);
      const uint32_t e = uint32_t(d[0]) > uint32_t(d[1]) ? uint32_t(d[0]) : uint32_t(d[1]);
      if ((t & 63) < 16) col_part[t >> 6][c16 * 8 + i] = __uint_as_float(e);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const ScalePair sp = scale_from_amax_bits<MODE>(row16_max_u32(__float_as_uint(max_abs8(v[j]))));
      *reinterpret_cast<uint2*>(p.q + (row0 + j) * p.ld_q + col) =
          uint2{quant4(v[j][0], v[j][1], v[j][2], v[j][3], sp.inv), quant4(v[j][4], v[j][5], v[j][6], v[j][7], sp.inv)};
      if (c16 == 0) p.scales[bc * mp + row0 + j] = sp.s;
    }
    __syncthreads();
    if (t < 128) {
      float m = col_part[0][t];
#pragma unroll
      for (int k = 1; k < 8; ++k) m = __builtin_fmaxf(m, col_part[k][t]);
      const ScalePair sc = scale_from_amax_bits<MODE>(__float_as_uint(m));
      inv_col[t] = sc.inv;
      p.scales_t[br * p.D + bc * 128 + t] = sc.s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      tile[((c16 * 8 + i) * kPitch + rq * 4) >> 2] = quant4(v[0][i], v[1][i], v[2][i], v[3][i], inv_col[c16 * 8 + i]);
    __syncthreads();
    const int cc = t >> 2, hh = t & 3;
    const uint32_t* src = tile + ((cc * kPitch + hh * 32) >> 2);
    uint8_t* dst = p.q_t + (bc * 128 + cc) * p.ld_qt + br * 128 + hh * 32;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      reinterpret_cast<u32x4*>(dst)[k] = u32x4{src[4 * k], src[4 * k + 1], src[4 * k + 2], src[4 * k + 3]};
    // the next block's writes of col_part come after its last reader's barrier, those of inv_col and tile after two
    // more; the tile's readers above are behind the first of them
  }
}

template <typename T, typename W, int TPR, int R, int OUT>
hipError_t launch_rows(const NormArgs& p, hipStream_t st) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  const dim3 grid(grid_of((p.M - 1) / RPB + 1, NT));
  // The second pass over both tilings reads h again, which is x where there is no residual.
  if (p.once && (p.r || OUT != kOutNone)) hipLaunchKernelGGL((rmsnorm_kernel<T, W, TPR, R, OUT, true>), grid, dim3(NT), 0, st, p);
  else hipLaunchKernelGGL((rmsnorm_kernel<T, W, TPR, R, OUT, false>), grid, dim3(NT), 0, st, p);
  return hipGetLastError();
}

// A row's threads by its width.  Measured (8192x7168 BF16 with a residual, FP8, us): 256 threads of 4 runs 78, 512 of 2
// 83, 1024 of 1 106; 8192x2048: 256 of 1 22.8, 64 of 4 23.4; 65536x128: 16 lanes of 1 14.0, 64 29.8; 65536x256: 16 of 2
// 21.6, 64 of 1 29.9 (all alone; a call among others takes 11.7 and 19.9 of the last two, and 8.1 and 11.7 without a
// residual, of which the vector units issue for 5.9 and 8.3).
template <typename T, typename W, int OUT>
hipError_t launch_out(const NormArgs& p, hipStream_t st) {
  if (p.D <= 128) return launch_rows<T, W, 16, 1, OUT>(p, st);
  if (p.D <= 256) return launch_rows<T, W, 16, 2, OUT>(p, st);
  if (p.D <= 512) return launch_rows<T, W, 64, 1, OUT>(p, st);
  if (p.D <= 1024) return launch_rows<T, W, 64, 2, OUT>(p, st);
  if (p.D <= 2048) return launch_rows<T, W, 256, 1, OUT>(p, st);
  if (p.D <= 4096) return launch_rows<T, W, 256, 2, OUT>(p, st);
  if (p.D <= 8192) return launch_rows<T, W, 256, 4, OUT>(p, st);
  if (p.D <= 16384) return launch_rows<T, W, 1024, 2, OUT>(p, st);
  return launch_rows<T, W, 1024, 4, OUT>(p, st);
}

template <typename T, typename W>
hipError_t launch_fp8(const NormArgs& p, int mode, hipStream_t st) {
  if (!p.q_t) return mode == kModePow2 ? launch_out<T, W, kOutFp8Pow2>(p, st) : launch_out<T, W, kOutFp8>(p, st);
  const hipError_t e = launch_out<T, W, kOutNone>(p, st);
  if (e != hipSuccess) return e;
  NormArgs d = p;
  if (!p.r) d.h = const_cast<void*>(p.x), d.ld_h = p.ld_x;
  const dim3 grid(grid_of((p.D / 128) * ((p.M + 127) / 128), 512));
  if (mode == kModePow2) hipLaunchKernelGGL((rmsnorm_dual_kernel<T, W, kModePow2>), grid, dim3(512), 0, st, d);
  else hipLaunchKernelGGL((rmsnorm_dual_kernel<T, W, kModeMaxAbs>), grid, dim3(512), 0, st, d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_rmsnorm(const NormArgs& p, bool x_bf16, bool w_bf16, int mode, hipStream_t st) {
  if (x_bf16) return w_bf16 ? launch_fp8<uint16_t, uint16_t>(p, mode, st) : launch_fp8<uint16_t, float>(p, mode, st);
  return w_bf16 ? launch_fp8<float, uint16_t>(p, mode, st) : launch_fp8<float, float>(p, mode, st);
}

hipError_t launch_int8_rmsnorm(const NormArgs& p, bool x_bf16, bool w_bf16, hipStream_t st) {
  if (x_bf16)
    return w_bf16 ? launch_out<uint16_t, uint16_t, kOutInt8>(p, st) : launch_out<uint16_t, float, kOutInt8>(p, st);
  return w_bf16 ? launch_out<float, uint16_t, kOutInt8>(p, st) : launch_out<float, float, kOutInt8>(p, st);
}

}  // namespace fp8q
