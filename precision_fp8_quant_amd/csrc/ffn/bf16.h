// BF16 and FP32 rows of eight elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8q {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Two floats rounded to nearest-even BF16, a in the low half
// (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2b));
}

// Eight consecutive elements as they lie in memory.
template <typename T> struct Row8;
template <> struct Row8<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ void zero() { w = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
};
template <> struct Row8<float> {
  v4f a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const v4f*>(p)[0];
    b = reinterpret_cast<const v4f*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = v4f{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p) =
      u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<v4f*>(p)[0] = v4f{v[0], v[1], v[2], v[3]};
  reinterpret_cast<v4f*>(p)[1] = v4f{v[4], v[5], v[6], v[7]};
}

}  // namespace fp8q
