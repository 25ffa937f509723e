// 8-bit integer codes with one scale for each row.
//
//   a = max(max_k |x[r][k]|, 127 * 2^-126)
//   s = fl32(a * fl32(1/127)), inv = fl32(127 * fl32(1/a))
//   q = rne(fl32(x * inv))
// (products with reciprocals rather than quotients: what a caller who writes the
// rule with tensors gets, so that codes agree to the last one.)
// |x| <= a and inv < (127 / a)(1 + 2^-20) keep |x inv| below 127.5, so the
// rounded code needs no clamp.
//
// A streaming pass: a row is read once, held in registers between its maximum
// and its codes, and written as 8 codes per lane.  TPR threads share a row (a
// DPP row of 16, a wave, or the 256-thread workgroup) and hold R runs of 8 elements each; rows
// longer than that are read twice.
#include "../fp8q_device.h"
#include "bf16.h"
#include "ffn_launch.h"

namespace fp8q {
namespace {

constexpr uint32_t kInt8FloorBits = 0x03FE0000u;   // 127 * 2^-126

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// Code in the low byte: adding 1.5 * 2^23 rounds to nearest-even in units of
// one and leaves the integer's two's complement in the low mantissa bits.
__device__ __forceinline__ uint32_t code(float x, float inv) { return __float_as_uint(x * inv + 12582912.0f); }

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(b, a, 0x0C0C0400u) | __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
}

// The columns [col, col + 8) of a row of `cols`, zeros beyond its end.
template <typename T>
__device__ __forceinline__ void load_run(const T* row, int64_t col, int64_t cols, float (&v)[8]) {
  if (col + 8 <= cols) {
    Row8<T> x;
    x.load(row + col);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x.get(i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? load1(row + col + i) : 0.0f;
  }
}

__device__ __forceinline__ void store_run(int8_t* row, int64_t col, int64_t cols, const float (&v)[8], float inv) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code(v[i], inv);
  if (col + 8 <= cols) {
    *reinterpret_cast<uint2*>(row + col) = uint2{pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) row[col + i] = int8_t(c[i]);
  }
}

__device__ __forceinline__ float run_max(float m, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
  return m;
}

// Max over the row's threads, in every thread.
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* wave_max) {
  uint32_t m = row16_max_u32(__float_as_uint(v));
  if constexpr (TPR == 16) return __builtin_fmaxf(__uint_as_float(m), __uint_as_float(kInt8FloorBits));
  const auto a = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  const uint32_t y = uint32_t(a[0]) > uint32_t(a[1]) ? uint32_t(a[0]) : uint32_t(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  m = uint32_t(b[0]) > uint32_t(b[1]) ? uint32_t(b[0]) : uint32_t(b[1]);
  float r = __uint_as_float(m);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = r;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) r = __builtin_fmaxf(r, wave_max[w]);
    __syncthreads();                               // wave_max is reused by the next row
  }
  return __builtin_fmaxf(r, __uint_as_float(kInt8FloorBits));
}

// R > 0: a row of at most 8 R TPR elements in registers.  R == 0: any length,
// read twice.
template <typename T, int TPR, int R>
__global__ __launch_bounds__(256) void int8_quant_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                              int64_t ld_x, int8_t* __restrict__ q, int64_t ld_q,
                                                              float* __restrict__ scales) {
  __shared__ float wave_max[4];
  constexpr int RPB = 256 / TPR;                   // rows per workgroup
  const int t = threadIdx.x & (TPR - 1);
  const int64_t step = int64_t(gridDim.x) * RPB;
  // uniform over the TPR threads of a row: barriers (TPR 256) and lane exchanges stay matched
  for (int64_t r = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR; r < rows; r += step) {
    const T* src = x + r * ld_x;
    int8_t* dst = q + r * ld_q;
    if constexpr (R > 0) {
      float v[R][8], m = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) load_run(src, int64_t(i * TPR + t) * 8, cols, v[i]);
#pragma unroll
      for (int i = 0; i < R; ++i) m = run_max(m, v[i]);
      const float a = row_max<TPR>(m, wave_max);
      const float inv = (1.0f / a) * 127.0f;
      if (t == 0) scales[r] = a * (1.0f / 127.0f);
#pragma unroll
      for (int i = 0; i < R; ++i) store_run(dst, int64_t(i * TPR + t) * 8, cols, v[i], inv);
    } else {
      float m = 0.0f;
      for (int64_t c = t * 8; c < cols; c += TPR * 8) {
        float v[8];
        load_run(src, c, cols, v);
        m = run_max(m, v);
      }
      const float a = row_max<TPR>(m, wave_max);
      const float inv = (1.0f / a) * 127.0f;
      if (t == 0) scales[r] = a * (1.0f / 127.0f);
      for (int64_t c = t * 8; c < cols; c += TPR * 8) {
        float v[8];
        load_run(src, c, cols, v);
        store_run(dst, c, cols, v, inv);
      }
    }
  }
}

template <typename T, int TPR, int R>
hipError_t launch_cfg(const T* x, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q, int64_t ld_q, float* scales,
                      hipStream_t st) {
  constexpr int RPB = 256 / TPR;
  const int64_t blocks = (rows - 1) / RPB + 1;
  hipLaunchKernelGGL((int8_quant_rows_kernel<T, TPR, R>), dim3(grid_of(blocks, 256)), dim3(256), 0, st, x, rows, cols, ld_x,
                     q, ld_q, scales);
  return hipGetLastError();
}

// Up to 128 elements 16 lanes per row, up to 1024 a wave, the workgroup beyond.
// Measured in BF16: 65536x100 17.7 us with a wave per row, 11.9 with 16 lanes (a call);
// 65536x512 18.0 us (5.6 TB/s), 8192x7168 37 us (4.8), 8192x18432 93 us (4.9,
// 228 when the row was read twice); FP32 18432x7168 120 us (5.5).
template <typename T>
hipError_t launch(const T* x, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q, int64_t ld_q, float* scales,
                  hipStream_t st) {
  if (cols <= 128) return launch_cfg<T, 16, 1>(x, rows, cols, ld_x, q, ld_q, scales, st);
  if (cols <= 512) return launch_cfg<T, 64, 1>(x, rows, cols, ld_x, q, ld_q, scales, st);
  if (cols <= 1024) return launch_cfg<T, 64, 2>(x, rows, cols, ld_x, q, ld_q, scales, st);
  if (cols <= 2048) return launch_cfg<T, 256, 1>(x, rows, cols, ld_x, q, ld_q, scales, st);
  if (cols <= 4096) return launch_cfg<T, 256, 2>(x, rows, cols, ld_x, q, ld_q, scales, st);
  if (cols <= 8192) return launch_cfg<T, 256, 4>(x, rows, cols, ld_x, q, ld_q, scales, st);
  if (cols <= 20480) return launch_cfg<T, 256, 10>(x, rows, cols, ld_x, q, ld_q, scales, st);
  return launch_cfg<T, 256, 0>(x, rows, cols, ld_x, q, ld_q, scales, st);
}

}  // namespace

hipError_t launch_int8_quant_rows(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q,
                                  int64_t ld_q, float* scales, hipStream_t st) {
  return bf16 ? launch(static_cast<const uint16_t*>(x), rows, cols, ld_x, q, ld_q, scales, st)
              : launch(static_cast<const float*>(x), rows, cols, ld_x, q, ld_q, scales, st);
}

}  // namespace fp8q
