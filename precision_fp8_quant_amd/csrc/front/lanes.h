// Sums and maxima over groups of lanes, the same in every lane of the group.
// Groups of 8 and 16 go by DPP (quad permutes, then the mirrors of a half row
// and of a row), 32 and 64 by the gfx950 permlane swaps.  Every lane of the
// wave must be active.
#pragma once

#include "../fp8q_device.h"

namespace fp8q {

// What lanes of the wave wrote to LDS before it is there for those that read
// behind it: LDS keeps a wave's order, the compiler has to.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  asm volatile("" ::: "memory");
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xF, 0xF, true));
}

// op(float bits, float bits) -> float bits, commutative
template <int N, typename Op>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, Op op) {
  static_assert(N == 8 || N == 16 || N == 32 || N == 64, "group sizes with a reduction of their own");
  v = op(v, dpp<0xB1>(v));                         // quad_perm [1,0,3,2]
  v = op(v, dpp<0x4E>(v));                         // quad_perm [2,3,0,1]
  v = op(v, dpp<0x141>(v));                        // row_half_mirror
  if constexpr (N >= 16) v = op(v, dpp<0x140>(v)); // row_mirror
  if constexpr (N >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(uint32_t(a[0]), uint32_t(a[1]));
  }
  if constexpr (N >= 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(uint32_t(a[0]), uint32_t(a[1]));
  }
  return v;
}

template <int N> __device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_reduce<N>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int N> __device__ __forceinline__ float lanes_max(float v) {
  return __uint_as_float(lanes_reduce<N>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int N> __device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v) {
  return lanes_reduce<N>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int N> __device__ __forceinline__ uint32_t lanes_min_u32(uint32_t v) {
  return lanes_reduce<N>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// v summed over the lanes that have the same place in their group of N, in each of them.
template <int N>
__device__ __forceinline__ float groups_sum(float v) {
  if constexpr (N <= 8) v += __uint_as_float(dpp<0x128>(__float_as_uint(v)));        // row_ror by 8: the other half row
  if constexpr (N <= 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(uint32_t(a[0])) + __uint_as_float(uint32_t(a[1]));
  }
  if constexpr (N <= 32) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(uint32_t(a[0])) + __uint_as_float(uint32_t(a[1]));
  }
  return v;
}

// Sum over the TPR threads that share a row: a group of lanes, a wave, or TPR / 64
// waves of the workgroup through `part`, one word per wave.  With TPR > 64 every
// thread of the workgroup calls it; `part` may be written again after the next
// barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = lanes_sum<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    const float* mine = part + threadIdx.x / TPR * (TPR / 64);
    v = mine[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += mine[w];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* part) {
  v = lanes_max<(TPR < 64 ? TPR : 64)>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = __builtin_fmaxf(v, part[w]);
  }
  return v;
}

}  // namespace fp8q
