// Gradient of h = act(g) * u, quantized in both tilings in one pass.
//
//   dg = dh u act'(g),  du = dh act(g),  D = [dg | du]
//   act(g) = g s, act'(g) = s + g s (1 - s) t'(g), s = sigma(t(g))   (gate_act.h)
// D's 1x128 tiles (Dgrad's operand) and transposed 128x1 tiles (Wgrad's) are
// quantized from the FP32 values by the rule of include/fp8q.h; D itself goes
// to memory only where the caller asks for it.
//
// A streaming pass (6 bytes in, 4.06 out per element of dh in BF16) whose
// arithmetic comes close to the memory's time: some forty vector operations
// per element.  One 512-thread workgroup per 128 x 128 block of dh, which
// gives one block of dg and one of du.  Thread t owns columns 8*(t%16)..+7 of
// rows 4*(t/16)..+3, so a DPP row of 16 lanes holds a 1x128 tile.
//   1. dg and du of the thread's 4 x 8 elements
//   2. 1x128: max over the DPP row for each of the 8 (half, row) tiles; lane i
//      of the DPP row derives the scales of tile i alone and the others take
//      them by row broadcasts; row-major codes
//   3. 128x1: the thread's column maxima over its 4 rows meet in LDS, where 256
//      threads finish one column each (32 partials, scale pair)
//   4. transposed codes staged in LDS (over the partials) and copied out as 32
//      bytes of one column at a time.
// 2 workgroups per CU (at most 128 registers) let one's memory run beside the
// other's arithmetic and barriers.  Measured on 8192x18432, SiLU, BF16: 306 us,
// 5.0 TB/s (a large copy: 4.9); 562 us with every lane deriving every scale and
// one workgroup per CU; 351 us with non-temporal stores; 391 us held to 5 waves
// per SIMD (spills).
// Rows past M are zeros, so the outputs cover whole 128-row tiles.
#include "../fp8q_device.h"
#include "bf16.h"
#include "ffn_launch.h"

namespace fp8q {
namespace {

constexpr int kPitch = 132;    // bytes per LDS row of the transposed tile

struct BwdArgs {
  int64_t M, F;
  int64_t ld_dh, ld_gu;
  uint8_t* q; int64_t ld_q; float* scales;
  uint8_t* q_t; int64_t ld_qt; float* scales_t;
  int64_t ld_dgu;
  float c1, c3;
};

// dg and du of one element.  x = -t log2(e) is held at 126, so e = 2^x cannot
// overflow: s = 1 / (1 + e) and 1 - s = e s keep their digits on both sides,
// and where x is held (s = 2^-126) g is held at -128, which keeps g s under
// 2^-118 for every g.
__device__ __forceinline__ void grad(float dh, float g, float u, float c1, float c3, float& dg, float& du) {
  const float g2 = __builtin_fminf(g * g, 1.0e4f);
  const float x = -1.44269504088896341f * (g * __builtin_fmaf(c3, g2, c1));
  const float e = __builtin_amdgcn_exp2f(__builtin_fminf(x, 126.0f));
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  const float gs = __builtin_fmaxf(g, -128.0f) * s;
  const float slope = __builtin_fmaf(gs * (e * s), __builtin_fmaf(3.0f * c3, g2, c1), s);
  dg = dh * u * slope;
  du = dh * gs;
}

// A product of |x| <= a with inv <= (448 / a)(1 + 2^-24) rounds to at most the
// code of 448, so no clamp is needed before the conversion.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

__device__ __forceinline__ float max_abs(float m, float v) { return __builtin_fmaxf(m, __builtin_fabsf(v)); }

template <int LANE>
__device__ __forceinline__ float row_bcast(float v) {       // lane LANE of every DPP row of 16, to the whole row
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x150 + LANE, 0xF, 0xF, true));
}

template <typename T, int MODE>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4, 8)))
void gated_backward_kernel(const T* __restrict__ dh, const T* __restrict__ gu, T* __restrict__ dgu, BwdArgs p) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[256 * kPitch / 4];   // column maxima [2][32][128], then the tiles
  __shared__ __attribute__((aligned(16))) float inv_col[256];
  static_assert(sizeof(lds) >= 2 * 32 * 128 * 4, "the column maxima fit under the transposed tiles");
  const int t = threadIdx.x;
  const int c16 = t & 15, rq = t >> 4;
  const int64_t cblocks = p.F >> 7, rblocks = (p.M + 127) >> 7;
  const int64_t mp = rblocks << 7, f2 = 2 * p.F;
  for (int64_t blk = blockIdx.x; blk < cblocks * rblocks; blk += gridDim.x) {   // block-uniform: barriers stay matched
    // Column-major: consecutive workgroups extend the same 256 runs of q_t, which
    // leave in 128-byte pieces (8192x18432: 323 -> 306 us against row-major).
    const int64_t br = blk % rblocks, bc = blk / rblocks;
    const int64_t col = bc * 128 + c16 * 8;
    const int64_t row0 = br * 128 + rq * 4;
    float d[2][4][8];                              // dg, du of the thread's 4 rows x 8 columns
    constexpr int ROWS = sizeof(T) == 2 ? 4 : 2;
    const T* ph = dh + row0 * p.ld_dh + col;
    const T* pg = gu + row0 * p.ld_gu + col;
    T* pd = dgu ? dgu + row0 * p.ld_dgu + col : nullptr;
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += ROWS) {
      Row8<T> vh[ROWS], vg[ROWS], vu[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int64_t r = row0 + j0 + j;
        if (r < p.M) {
          vh[j].load(ph);
          vg[j].load(pg);
          vu[j].load(pg + p.F);
        } else {
          vh[j].zero();
          vg[j].zero();
          vu[j].zero();
        }
        ph += p.ld_dh;
        pg += p.ld_gu;
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          grad(vh[j].get(i), vg[j].get(i), vu[j].get(i), p.c1, p.c3, d[0][j0 + j][i], d[1][j0 + j][i]);
      if (dgu) {
#pragma unroll
        for (int j = j0; j < j0 + ROWS; ++j, pd += p.ld_dgu)
          if (row0 + j < p.M) {
            store8(pd, d[0][j]);
            store8(pd + p.F, d[1][j]);
          }
      }
      asm volatile("" ::: "memory");               // the next rows are not loaded before: registers
    }

    // 128x1 partial maxima first: their barrier is then met while the row codes are on their way
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        m[i] = max_abs(max_abs(max_abs(__builtin_fabsf(d[half][0][i]), d[half][1][i]), d[half][2][i]), d[half][3][i]);
      v4f* dst = reinterpret_cast<v4f*>(lds + (half * 32 + rq) * 128 + c16 * 8);
      dst[0] = v4f{m[0], m[1], m[2], m[3]};
      dst[1] = v4f{m[4], m[5], m[6], m[7]};
    }

    // 1x128: tile i of the DPP row is (half i/4, row i%4)
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float(&v)[8] = d[i >> 2][i & 3];
      float m = __builtin_fabsf(v[0]);
#pragma unroll
      for (int k = 1; k < 8; ++k) m = max_abs(m, v[k]);
      const uint32_t b = row16_max_u32(__float_as_uint(m));
      mine = (c16 & 7) == i ? b : mine;
    }
    const ScalePair sp = scale_from_amax_bits<MODE>(mine);
    if (c16 < 8) p.scales[((c16 >> 2) * cblocks + bc) * mp + row0 + (c16 & 3)] = sp.s;
    auto row_codes = [&](int i, float inv) {
      const float(&v)[8] = d[i >> 2][i & 3];
      *reinterpret_cast<uint2*>(p.q + (row0 + (i & 3)) * p.ld_q + (i >> 2) * p.F + col) =
          uint2{quant4(v[0], v[1], v[2], v[3], inv), quant4(v[4], v[5], v[6], v[7], inv)};
    };
    row_codes(0, row_bcast<0>(sp.inv));
    row_codes(1, row_bcast<1>(sp.inv));
    row_codes(2, row_bcast<2>(sp.inv));
    row_codes(3, row_bcast<3>(sp.inv));
    row_codes(4, row_bcast<4>(sp.inv));
    row_codes(5, row_bcast<5>(sp.inv));
    row_codes(6, row_bcast<6>(sp.inv));
    row_codes(7, row_bcast<7>(sp.inv));
    __syncthreads();

    if (t < 256) {
      const int half = t >> 7, c = t & 127;
      const float* part = reinterpret_cast<const float*>(lds) + half * 32 * 128 + c;
      float m = part[0];
#pragma unroll
      for (int k = 1; k < 32; ++k) m = __builtin_fmaxf(m, part[k * 128]);
      const ScalePair sc = scale_from_amax_bits<MODE>(__float_as_uint(m));
      inv_col[t] = sc.inv;
      p.scales_t[br * f2 + half * p.F + bc * 128 + c] = sc.s;
    }
    __syncthreads();

#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float inv[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const v4f x = *reinterpret_cast<const v4f*>(inv_col + half * 128 + c16 * 8 + 4 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) inv[4 * k + i] = x[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        lds[((half * 128 + c16 * 8 + i) * kPitch + rq * 4) >> 2] =
            quant4(d[half][0][i], d[half][1][i], d[half][2][i], d[half][3][i], inv[i]);
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int cc = t >> 2, hh = t & 3;
      const uint32_t* src = lds + (((half * 128 + cc) * kPitch + hh * 32) >> 2);
      uint8_t* dst = p.q_t + (half * p.F + bc * 128 + cc) * p.ld_qt + br * 128 + hh * 32;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        reinterpret_cast<u32x4*>(dst)[k] = u32x4{src[4 * k], src[4 * k + 1], src[4 * k + 2], src[4 * k + 3]};
    }
    __syncthreads();                               // the LDS is reused by the next block
  }
}

}  // namespace

hipError_t launch_gated_backward(float act_c1, float act_c3, int64_t M, int64_t F, const void* dh, int64_t ld_dh,
                                 const void* gu, int64_t ld_gu, bool bf16, int mode, uint8_t* q, int64_t ld_q,
                                 float* scales, uint8_t* q_t, int64_t ld_qt, float* scales_t, void* dgu,
                                 int64_t ld_dgu, hipStream_t st) {
  const BwdArgs p{M, F, ld_dh, ld_gu, q, ld_q, scales, q_t, ld_qt, scales_t, ld_dgu, act_c1, act_c3};
  const dim3 grid(grid_of((F / 128) * ((M + 127) / 128), 512));
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
