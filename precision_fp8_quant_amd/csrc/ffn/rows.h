// Rows of any length, eight elements at a time, and 8-bit integer codes.
#pragma once

#include "bf16.h"

namespace fp8q {

constexpr uint32_t kInt8FloorBits = 0x03FE0000u;   // 127 * 2^-126

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// 8-bit integer code in the low byte: adding 1.5 * 2^23 rounds to nearest-even in units of
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

}  // namespace fp8q
