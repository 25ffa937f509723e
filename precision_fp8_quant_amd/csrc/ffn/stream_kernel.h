// Products of 8-bit operands for few rows of A: the weight streams once from
// memory straight into matrix-instruction registers.
//
//   plain:  C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k] (+ bias[n])
//   gated:  h[m][f] = act(g) u,  g from B's rows [0, N), u from rows [N, 2N)
// with 8-bit integers (32-bit integer sums, scales per row of A and B) or
// block-scaled FP8 (one FP32 promotion per 128-deep K-group with that group's
// scales, as in gemm_kernel.h).
//
// For M rows the weight's K N bytes are read once and feed 2 M operations
// each, so below some tens of rows the memory bounds the product and all that
// counts is how many bytes of B are in flight.  A workgroup of 8 waves owns
// 16 MF rows x 16 columns (gated: of both projections); the waves share out K
// in runs of UNROLL 128-byte groups, and each loads its B bytes from global
// memory directly in fragment order: no LDS and no barrier stands between the
// loads and the matrix instructions.  The waves' partial sums meet in LDS
// once, at the end, and are added in a fixed order, so the result does not
// depend on timing.
//
// The matrix instruction takes the B fragment as source A (16 rows of N) and
// the A fragment as source B (16 rows of M), so a lane's four results are four
// consecutive columns of one row.  The K order within a group is free as long
// as both operands agree: lane quarter q holds bytes [16q, 16q+16) and
// [64+16q, 64+16q+16) of its row's 128.
#pragma once

#include "../gemm_kernel.h"
#include "ffn_launch.h"
#include "gate_act.h"

namespace fp8q {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kStreamWaves = 8;
constexpr int64_t kStreamRows = 64;    // rows of A up to which the weight is streamed

struct Frag {
  u32x4 lo, hi;
};

// 16 bytes of a row whose first `left` bytes are inside K: the rest is zero.
__device__ __forceinline__ u32x4 mask_bytes(u32x4 v, int64_t left) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int64_t n = left - 4 * w;               // bytes of word w inside K
    if (n <= 0) v[w] = 0u;
    else if (n < 4) v[w] &= (1u << (8 * int(n))) - 1u;
  }
  return v;
}

// Bytes [k, k+16) and [k+64, k+80) of a row.  TAIL: the group reaches beyond
// K; chunks wholly outside are not read, and with MASK a chunk's bytes beyond
// K are cleared (one operand is enough: 0 times any integer is 0).
template <bool TAIL, bool MASK>
__device__ __forceinline__ Frag load_frag(const uint8_t* row, int64_t k, int64_t K) {
  Frag f;
  if constexpr (!TAIL) {
    f.lo = *reinterpret_cast<const u32x4*>(row + k);
    f.hi = *reinterpret_cast<const u32x4*>(row + k + 64);
  } else {
    f.lo = f.hi = u32x4{0u, 0u, 0u, 0u};
    if (k < K) f.lo = *reinterpret_cast<const u32x4*>(row + k);
    if (k + 64 < K) f.hi = *reinterpret_cast<const u32x4*>(row + k + 64);
    if constexpr (MASK) {
      f.lo = mask_bytes(f.lo, K - k);
      f.hi = mask_bytes(f.hi, K - k - 64);
    }
  }
  return f;
}

template <bool INT8, bool GATED, int MF, int OUT>
__global__ __launch_bounds__(kStreamWaves * 64) void stream_kernel(FfnArgs p) {
  constexpr int NP = GATED ? 2 : 1;               // projections
  constexpr int UNROLL = MF <= 2 ? 4 : 2;         // 128-byte groups loaded before the first is used
  typedef typename std::conditional<INT8, v4i, v4f>::type acc_t;
  __shared__ acc_t part[kStreamWaves][NP * MF][64];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t ntiles = (p.N + 15) >> 4;
  const int64_t n0 = (blockIdx.x % ntiles) * 16;
  const int64_t m0 = (blockIdx.x / ntiles) * (16 * MF);

  // Rows past the end repeat the last one: their products are not stored.
  const uint8_t* arow[MF];
  const uint8_t* brow[NP];
  int64_t mrow[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t m = m0 + 16 * i + lr;
    mrow[i] = m < p.M ? m : p.M - 1;
    arow[i] = p.a + mrow[i] * p.lda + 16 * lq;
  }
  {
    const int64_t n = n0 + lr < p.N ? n0 + lr : p.N - 1;
#pragma unroll
    for (int b = 0; b < NP; ++b) brow[b] = p.b + (b * p.N + n) * p.ldb + 16 * lq;
  }

  acc_t acc[NP][MF];
#pragma unroll
  for (int b = 0; b < NP; ++b)
#pragma unroll
    for (int i = 0; i < MF; ++i) acc[b][i] = acc_t{0, 0, 0, 0};

  const int64_t KG = (p.K + 127) >> 7;            // FP8: K is a multiple of 128
  const int64_t kfull = p.K >> 7;                 // groups wholly inside K

  auto use = [&](const Frag (&fa)[MF], const Frag (&fb)[NP], int64_t g) {
    if constexpr (INT8) {
#pragma unroll
      for (int b = 0; b < NP; ++b)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          acc[b][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, fb[b].lo),
                                                            __builtin_bit_cast(v4i, fa[i].lo), acc[b][i], 0, 0, 0);
          acc[b][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, fb[b].hi),
                                                            __builtin_bit_cast(v4i, fa[i].hi), acc[b][i], 0, 0, 0);
        }
    } else {
      const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int b = 0; b < NP; ++b) {
        const float sb = p.sb[((b * p.N + n0) >> 7) * KG + g];
        const v8i vb = {int(fb[b].lo.x), int(fb[b].lo.y), int(fb[b].lo.z), int(fb[b].lo.w),
                        int(fb[b].hi.x), int(fb[b].hi.y), int(fb[b].hi.z), int(fb[b].hi.w)};
#pragma unroll
        for (int i = 0; i < MF; ++i) {
          const v8i va = {int(fa[i].lo.x), int(fa[i].lo.y), int(fa[i].lo.z), int(fa[i].lo.w),
                          int(fa[i].hi.x), int(fa[i].hi.y), int(fa[i].hi.z), int(fa[i].hi.w)};
          const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, zero, 0, 0, 0, 0, 0, 0);
          const float c = p.sa[g * p.M + mrow[i]] * sb;
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[b][i][j] = __builtin_fmaf(d[j], c, acc[b][i][j]);
        }
      }
    }
  };

  int64_t g = wave * UNROLL;
  for (; g + UNROLL <= kfull; g += kStreamWaves * UNROLL) {
    Frag fa[UNROLL][MF], fb[UNROLL][NP];
#pragma unroll
    for (int s = 0; s < UNROLL; ++s) {
#pragma unroll
      for (int b = 0; b < NP; ++b) fb[s][b] = load_frag<false, false>(brow[b], (g + s) * 128, p.K);
#pragma unroll
      for (int i = 0; i < MF; ++i) fa[s][i] = load_frag<false, false>(arow[i], (g + s) * 128, p.K);
    }
#pragma unroll
    for (int s = 0; s < UNROLL; ++s) use(fa[s], fb[s], g + s);
  }
  // the run that holds the last whole groups and the group that reaches beyond K
  for (int64_t e = g + UNROLL < KG ? g + UNROLL : KG; g < e; ++g) {
    Frag fa[MF], fb[NP];
    const int64_t left = p.K - 16 * lq;           // K as seen from this lane's first chunk
#pragma unroll
    for (int b = 0; b < NP; ++b) fb[b] = load_frag<true, false>(brow[b], g * 128, left);
#pragma unroll
    for (int i = 0; i < MF; ++i) fa[i] = load_frag<true, true>(arow[i], g * 128, left);
    use(fa, fb, g);
  }

#pragma unroll
  for (int b = 0; b < NP; ++b)
#pragma unroll
    for (int i = 0; i < MF; ++i) part[wave][b * MF + i][lane] = acc[b][i];
  __syncthreads();

  // Thread t adds the 8 waves' parts of fragment t/64, lane t%64, and finishes
  // four columns of one row.
  for (int f = wave; f < MF; f += kStreamWaves) {
    const int64_t m = m0 + 16 * f + lr;
    const int64_t n = n0 + 4 * lq;
    if (m >= p.M || n >= p.N) continue;
    acc_t sum[NP];
#pragma unroll
    for (int b = 0; b < NP; ++b) {
      sum[b] = part[0][b * MF + f][lane];
#pragma unroll
      for (int w = 1; w < kStreamWaves; ++w) sum[b] += part[w][b * MF + f][lane];
    }
    const int cols = p.N - n < 4 ? int(p.N - n) : 4;
    const float sa = (INT8 && p.K > 0) ? p.sa[m] : 1.0f;
    float y[NP][4], out[4];
#pragma unroll
    for (int b = 0; b < NP; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[b][j] = float(sum[b][j]);
        if constexpr (INT8) y[b][j] *= (p.K > 0 && j < cols) ? sa * p.sb[b * p.N + n + j] : 0.0f;
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (GATED) out[j] = gate_mul(y[0][j], y[1][j], p.act_c1, p.act_c3);
      else out[j] = (p.bias && j < cols) ? y[0][j] + p.bias[n + j] : y[0][j];
    }
    auto store = [&](void* base, int64_t ld, int64_t col, const float (&v)[4]) {
      if constexpr (OUT == kOutBF16) {
        uint16_t* dst = static_cast<uint16_t*>(base) + m * ld + col;
        if (cols == 4) {
          *reinterpret_cast<uint2*>(dst) = uint2{bf16_rne_bits(v[0]) | (bf16_rne_bits(v[1]) << 16),
                                                 bf16_rne_bits(v[2]) | (bf16_rne_bits(v[3]) << 16)};
        } else {
          for (int j = 0; j < cols; ++j) dst[j] = uint16_t(bf16_rne_bits(v[j]));
        }
      } else {
        float* dst = static_cast<float*>(base) + m * ld + col;
        if (cols == 4) *reinterpret_cast<v4f*>(dst) = v4f{v[0], v[1], v[2], v[3]};
        else
          for (int j = 0; j < cols; ++j) dst[j] = v[j];
      }
    };
    store(p.c, p.ldc, n, out);
    if constexpr (GATED)
      if (p.gu) {
        store(p.gu, p.ldgu, n, y[0]);
        store(p.gu, p.ldgu, p.N + n, y[1]);
      }
  }
}

template <bool INT8, bool GATED, int MF, int OUT>
static hipError_t launch_stream_cfg(const FfnArgs& p, hipStream_t st) {
  const int64_t tiles = ((p.N + 15) / 16) * ((p.M + 16 * MF - 1) / (16 * MF));
  hipLaunchKernelGGL((stream_kernel<INT8, GATED, MF, OUT>), dim3(unsigned(tiles)), dim3(kStreamWaves * 64), 0, st, p);
  return hipGetLastError();
}

template <bool INT8, bool GATED, int OUT>
static hipError_t launch_stream(const FfnArgs& p, hipStream_t st) {
  if (p.M <= 16) return launch_stream_cfg<INT8, GATED, 1, OUT>(p, st);
  if (p.M <= 32) return launch_stream_cfg<INT8, GATED, 2, OUT>(p, st);
  return launch_stream_cfg<INT8, GATED, 4, OUT>(p, st);
}

}  // namespace fp8q
