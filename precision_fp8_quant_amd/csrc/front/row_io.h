// A thread's runs of eight elements as they lie in memory, at rows whose
// length need not be a multiple of eight.
#pragma once

#include "../ffn/rows.h"

namespace fp8q {

__device__ __forceinline__ void put1(Row8<uint16_t>& x, int i, const uint16_t* p) {
  x.w[i >> 1] |= uint32_t(*p) << (16 * (i & 1));
}
__device__ __forceinline__ void put1(Row8<float>& x, int i, const float* p) {
  if (i < 4) x.a[i] = *p;
  else x.b[i - 4] = *p;
}

// Elements [col, col + 8) of a row of `cols`; zeros beyond its end.
template <typename T>
__device__ __forceinline__ void load_raw(Row8<T>& x, const T* row, int64_t col, int64_t cols) {
  if (col + 8 <= cols) {
    x.load(row + col);
  } else {
    x.zero();
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (col + i < cols) put1(x, i, row + col + i);
  }
}

__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = uint16_t(pack_bf16(v, 0.0f)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// v rounded to T, elements [col, col + 8) of a row of `cols`; nothing beyond its end.
template <typename T>
__device__ __forceinline__ void store_raw(T* row, int64_t col, int64_t cols, const float (&v)[8]) {
  if (col + 8 <= cols) {
    store8(row + col, v);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (col + i < cols) store1(row + col + i, v[i]);
  }
}

// What T holds of v.
__device__ __forceinline__ float held(float v, uint16_t) { return __uint_as_float(pack_bf16(v, 0.0f) << 16); }
__device__ __forceinline__ float held(float v, float) { return v; }

}  // namespace fp8q
