// Gradient of h = act(g) * u, quantized in both tilings in one pass.
//
//   dg = dh u act'(g),  du = dh act(g),  D = [dg | du]
//   (act' and its parts: gate_act.h)
// D's 1x128 tiles (Dgrad's operand) and transposed 128x1 tiles (Wgrad's) are
// quantized from the FP32 values by the rule of include/fp8q.h; D itself goes
// to memory only where the caller asks for it.
//
// One 512-thread workgroup per 128 x 128 block of dh, which gives one block of
// dg and one of du.  Thread t owns columns 8*(t%16)..+7 of rows 4*(t/16)..+3,
// so a DPP row of 16 lanes holds a 1x128 tile.  Each half of D goes through
// the same steps: row max over the DPP row, row-major codes; column max over
// the wave by the permlane swaps and over the waves through LDS; transposed
// codes staged in LDS and copied out as 32 bytes of one column per thread.
// Rows past M are zeros, so the outputs cover whole 128-row tiles.
#include "../fp8q_device.h"
#include "../gemm_kernel.h"
#include "ffn_launch.h"
#include "gate_act.h"

namespace fp8q {
namespace {

constexpr int kPitch = 132;    // bytes per LDS row of the transposed tile (conflict-free dword writes)

struct BwdArgs {
  int64_t M, F;
  int64_t ld_dh, ld_gu;
  uint8_t* q; int64_t ld_q; float* scales;
  uint8_t* q_t; int64_t ld_qt; float* scales_t;
  int64_t ld_dgu;
  float c1, c3;
};

// Eight consecutive values as FP32.
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const v4f a = reinterpret_cast<const v4f*>(p)[0], b = reinterpret_cast<const v4f*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[i + 4] = b[i];
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p) = u32x4{bf16_rne_bits(v[0]) | (bf16_rne_bits(v[1]) << 16),
                                       bf16_rne_bits(v[2]) | (bf16_rne_bits(v[3]) << 16),
                                       bf16_rne_bits(v[4]) | (bf16_rne_bits(v[5]) << 16),
                                       bf16_rne_bits(v[6]) | (bf16_rne_bits(v[7]) << 16)};
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<v4f*>(p)[0] = v4f{v[0], v[1], v[2], v[3]};
  reinterpret_cast<v4f*>(p)[1] = v4f{v[4], v[5], v[6], v[7]};
}

template <int MODE>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  a *= inv; b *= inv; c *= inv; d *= inv;
  if constexpr (MODE == kModeMaxAbs) {             // a power-of-two scale keeps every product within +-448
    a = clamp448(a); b = clamp448(b); c = clamp448(c); d = clamp448(d);
  }
  const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Max over lanes l, l^16, l^32, l^48.
__device__ __forceinline__ uint32_t rows4_max(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const uint32_t y = max_u32(uint32_t(a[0]), uint32_t(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return max_u32(uint32_t(b[0]), uint32_t(b[1]));
}

template <typename T, int MODE>
__global__ __launch_bounds__(512) void gated_backward_kernel(const T* __restrict__ dh, const T* __restrict__ gu,
                                                             T* __restrict__ dgu, BwdArgs p) {
  __shared__ uint32_t col_part[8][128];
  __shared__ uint32_t tile[128 * kPitch / 4];
  const int t = threadIdx.x;
  const int c16 = t & 15, rq = t >> 4, wave = t >> 6;
  const int64_t cblocks = p.F >> 7, rblocks = (p.M + 127) >> 7;
  const int64_t mp = rblocks << 7, f2 = 2 * p.F;
  for (int64_t blk = blockIdx.x; blk < cblocks * rblocks; blk += gridDim.x) {   // block-uniform: barriers stay matched
    const int64_t bc = blk % cblocks, br = blk / cblocks;
    const int64_t col = bc * 128 + c16 * 8;
    const int64_t row0 = br * 128 + rq * 4;
    float d[2][4][8];                              // dg, du of the thread's 4 rows x 8 columns
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = row0 + j;
      if (r < p.M) {
        float vh[8], vg[8], vu[8];
        load8(dh + r * p.ld_dh + col, vh);
        load8(gu + r * p.ld_gu + col, vg);
        load8(gu + r * p.ld_gu + p.F + col, vu);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const Gate e = gate_eval(vg[i], p.c1, p.c3);
          const float slope = __builtin_fmaf(vg[i] * (e.s * e.one_s), __builtin_fmaf(3.0f * p.c3, e.g2, p.c1), e.s);
          d[0][j][i] = vh[i] * vu[i] * slope;
          d[1][j][i] = vh[i] * (vg[i] * e.s);
        }
        if (dgu) {
          store8(dgu + r * p.ld_dgu + col, d[0][j]);
          store8(dgu + r * p.ld_dgu + p.F + col, d[1][j]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[0][j][i] = d[1][j][i] = 0.0f;
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t c0 = half * p.F + col;         // this thread's first column of D
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_u32(m, abs_bits(d[half][j][i]));
        const ScalePair sp = scale_from_amax_bits<MODE>(row16_max_u32(m));
        const float(&v)[8] = d[half][j];
        *reinterpret_cast<uint2*>(p.q + (row0 + j) * p.ld_q + c0) =
            uint2{quant4<MODE>(v[0], v[1], v[2], v[3], sp.inv), quant4<MODE>(v[4], v[5], v[6], v[7], sp.inv)};
        if (c16 == 0) p.scales[(c0 >> 7) * mp + row0 + j] = sp.s;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max_u32(m, abs_bits(d[half][j][i]));
        m = rows4_max(m);
        if ((t & 63) < 16) col_part[wave][c16 * 8 + i] = m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c16 * 8 + i;
        uint32_t m = col_part[0][c];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max_u32(m, col_part[w][c]);
        const ScalePair sp = scale_from_amax_bits<MODE>(m);
        if (rq == 0) p.scales_t[br * f2 + c0 + i] = sp.s;
        tile[(c * kPitch + rq * 4) >> 2] =
            quant4<MODE>(d[half][0][i], d[half][1][i], d[half][2][i], d[half][3][i], sp.inv);
      }
      __syncthreads();
      const int cc = t >> 2, hh = t & 3;
      const uint32_t* src = tile + ((cc * kPitch + hh * 32) >> 2);
      uint8_t* dst = p.q_t + (half * p.F + bc * 128 + cc) * p.ld_qt + br * 128 + hh * 32;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        reinterpret_cast<u32x4*>(dst)[k] = u32x4{src[4 * k], src[4 * k + 1], src[4 * k + 2], src[4 * k + 3]};
      __syncthreads();                             // col_part and tile are reused
    }
  }
}

}  // namespace

hipError_t launch_gated_backward(float act_c1, float act_c3, int64_t M, int64_t F, const void* dh, int64_t ld_dh,
                                 const void* gu, int64_t ld_gu, bool bf16, int mode, uint8_t* q, int64_t ld_q,
                                 float* scales, uint8_t* q_t, int64_t ld_qt, float* scales_t, void* dgu,
                                 int64_t ld_dgu, hipStream_t st) {
  const BwdArgs p{M, F, ld_dh, ld_gu, q, ld_q, scales, q_t, ld_qt, scales_t, ld_dgu, act_c1, act_c3};
  const int64_t blocks = (F / 128) * ((M + 127) / 128);
  const dim3 grid(unsigned(blocks < 0x7FFFFFFF ? blocks : 0x7FFFFFFF));
  auto go = [&](auto kernel, auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    hipLaunchKernelGGL(kernel, grid, dim3(512), 0, st, static_cast<const T*>(dh), static_cast<const T*>(gu),
                       static_cast<T*>(dgu), p);
    return hipGetLastError();
  };
  if (bf16)
    return mode == kModePow2 ? go(gated_backward_kernel<uint16_t, kModePow2>, (uint16_t*)nullptr)
                             : go(gated_backward_kernel<uint16_t, kModeMaxAbs>, (uint16_t*)nullptr);
  return mode == kModePow2 ? go(gated_backward_kernel<float, kModePow2>, (float*)nullptr)
                           : go(gated_backward_kernel<float, kModeMaxAbs>, (float*)nullptr);
}

}  // namespace fp8q
