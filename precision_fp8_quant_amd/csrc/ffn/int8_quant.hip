// 8-bit integer codes with one scale for each row.
//
//   a = max(max_k |x[r][k]|, 127 * 2^-126), s = fl32(a / 127), inv = fl32(127 / a)
//   q = rne(fl32(x * inv))
// |x| <= a and inv <= (127 / a)(1 + 2^-24) keep |x inv| below 127.5, so the
// rounded code needs no clamp.
#include "../fp8q_device.h"
#include "../gemm_kernel.h"
#include "ffn_launch.h"

namespace fp8q {
namespace {

constexpr uint32_t kInt8FloorBits = 0x03FE0000u;   // 127 * 2^-126

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// One 256-thread workgroup per row.
template <typename T>
__global__ __launch_bounds__(256) void int8_quant_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                              int64_t ld_x, int8_t* __restrict__ q, int64_t ld_q,
                                                              float* __restrict__ scales) {
  __shared__ uint32_t wave_max[4];
  const int t = threadIdx.x;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* src = x + r * ld_x;
    uint32_t m = kInt8FloorBits;
    for (int64_t c = t; c < cols; c += 256) {
      const uint32_t b = __float_as_uint(load1(src + c)) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
    for (int d = 32; d; d >>= 1) {
      const uint32_t o = uint32_t(__shfl_xor(int(m), d));
      m = o > m ? o : m;
    }
    if ((t & 63) == 0) wave_max[t >> 6] = m;
    __syncthreads();
    for (int w = 0; w < 4; ++w) m = wave_max[w] > m ? wave_max[w] : m;
    const float a = __uint_as_float(m);
    const float inv = 127.0f / a;
    if (t == 0) scales[r] = a / 127.0f;
    for (int64_t c = t; c < cols; c += 256) q[r * ld_q + c] = int8_t(int(__builtin_rintf(load1(src + c) * inv)));
    __syncthreads();                               // wave_max is reused by the next row
  }
}

}  // namespace

hipError_t launch_int8_quant_rows(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q,
                                  int64_t ld_q, float* scales, hipStream_t st) {
  const dim3 grid(unsigned(rows < 0x7FFFFFFF ? rows : 0x7FFFFFFF));
  if (bf16)
    hipLaunchKernelGGL((int8_quant_rows_kernel<uint16_t>), grid, dim3(256), 0, st, static_cast<const uint16_t*>(x),
                       rows, cols, ld_x, q, ld_q, scales);
  else
    hipLaunchKernelGGL((int8_quant_rows_kernel<float>), grid, dim3(256), 0, st, static_cast<const float*>(x), rows,
                       cols, ld_x, q, ld_q, scales);
  return hipGetLastError();
}

}  // namespace fp8q
