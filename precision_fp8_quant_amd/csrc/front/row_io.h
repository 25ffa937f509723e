// A thread's runs of eight elements as they lie in memory, at rows whose
// length need not be a multiple of eight.
#pragma once

#include "../ffn/rows.h"

namespace fp8q {

// The first n of the eight, zeros in place of the others.
__device__ __forceinline__ void keep(Row8<uint16_t>& x, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.w[i] = 2 * i + 1 < n ? x.w[i] : 2 * i < n ? x.w[i] & 0xFFFFu : 0u;
}
__device__ __forceinline__ void keep(Row8<float>& x, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.a[i] = i < n ? x.a[i] : 0.0f;
    x.b[i] = 4 + i < n ? x.b[i] : 0.0f;
  }
}
// ONCE: past the caches, for what nobody reads again.
template <bool ONCE, typename V>
__device__ __forceinline__ V load_vec(const void* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(static_cast<const V*>(p));
  else return *static_cast<const V*>(p);
}
template <bool ONCE>
__device__ __forceinline__ void load_chunks(Row8<uint16_t>& x, const uint16_t* p, int) { x.w = load_vec<ONCE, u32x4>(p); }
template <bool ONCE>
__device__ __forceinline__ void load_chunks(Row8<float>& x, const float* p, int n) {
  x.a = load_vec<ONCE, v4f>(p);
  if (n > 4) x.b = load_vec<ONCE, v4f>(p + 4);
}

// Elements [col, col + 8) of a row of `cols`, in two steps.  load_raw: rows are
// 16-byte aligned, and the 16 bytes that an element lies in are read whole; they
// are in one page.  trim: zeros for what the row does not own of them.  (One
// step would have the threads at a row's end wait for each of their loads.)
template <bool ONCE = false, typename T>
__device__ __forceinline__ void load_raw(Row8<T>& x, const T* row, int col, int cols) {
  x.zero();
  if (col < cols) load_chunks<ONCE>(x, row + col, cols - col);
}
template <typename T>
__device__ __forceinline__ void trim(Row8<T>& x, int col, int cols) {
  if (col + 8 > cols && col < cols) keep(x, cols - col);
}

__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = uint16_t(pack_bf16(v, 0.0f)); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// v rounded to T, elements [col, col + 8) of a row of `cols`; nothing beyond its end.
template <typename T>
__device__ __forceinline__ void store_raw(T* row, int col, int cols, const float (&v)[8]) {
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
