// Products of 8-bit operands for few rows of A: the weight streams once from
// memory straight into matrix-instruction registers.
//
//   plain:  C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k] (+ bias[n])
//   gated:  h[m][f] = act(g) u,  g from B's rows [0, N), u from rows [up, up + N)
// with 8-bit integers (32-bit integer sums, scales per row of A and B) or
// block-scaled FP8 (one FP32 promotion per 128-deep K-group with that group's
// scales, as in gemm_kernel.h).
//
// For M rows the weight's K N bytes are read once and feed 2 M operations
// each, so for few rows the memory bounds the product and all that counts is
// how many bytes of B are in flight.  A workgroup of 8 or 16 waves owns 16 MF
// rows x 16 NF columns (gated: of both projections); the waves share out K in
// contiguous runs, and each loads its B bytes from global memory directly in
// fragment order, UNROLL groups before the first is used: no LDS and no barrier
// stands between the loads and the matrix instructions.  The waves' partial
// sums meet in LDS once, at the end, and are added in a fixed order, so the
// result does not depend on timing.  Measured on one row: int8 gated
// 18432x7168 47.3 us (5.6 TB/s of weight), int8 7168x18432 26.0 us (5.1), FP8
// gated 18432x7168 47.3 us (5.6); the first 63.6 with the loads left to the
// compiler's order (three in flight) and the scales fetched in the epilogue.
//
// The matrix instruction takes the B fragment as source A (16 rows of N) and
// the A fragment as source B (16 rows of M), so a lane's four results are four
// consecutive columns of one row.  The K order within a group is free as long
// as both operands agree: lane quarter q holds bytes [16q, 16q+16) and
// [64+16q, 64+16q+16) of its row's 128.
#pragma once

#include "../gemm_kernel.h"
#include "bf16.h"
#include "ffn_launch.h"
#include "gate_act.h"

namespace fp8q {

typedef int v4i __attribute__((ext_vector_type(4)));

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

// HALF (gated): a workgroup owns 8 columns of h; rows 0 .. 7 of a B fragment are
// the gate's, rows 8 .. 15 the up projection's for the same columns.
template <bool INT8, bool GATED, bool HALF, int MF, int NF, int WAVES, int UNROLL, int OUT>
__global__ __launch_bounds__(WAVES * 64) void stream_kernel(FfnArgs p) {
  static_assert(!HALF || (GATED && NF == 1), "both projections in one fragment");
  constexpr int NP = GATED && !HALF ? 2 : 1;      // fragments of B per column fragment
  constexpr int NC = GATED ? 2 : 1;               // projections
  constexpr int CW = HALF ? 8 : 16 * NF;          // columns per workgroup
  typedef typename std::conditional<INT8, v4i, v4f>::type acc_t;
  __shared__ acc_t part[WAVES][NP * MF][64];
  __shared__ float s_sa[16 * MF], s_sb[NC * CW], s_bias[NC * CW];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t ntiles = (p.N + CW - 1) / CW;
  const int64_t n0 = (blockIdx.x % ntiles) * CW;
  const int64_t m0 = (blockIdx.x / ntiles) * (16 * MF);

  // Rows past the end repeat the last one: their products are not stored.
  const uint8_t* arow[MF];
  const uint8_t* brow[NP][NF];
  int64_t mrow[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t m = m0 + 16 * i + lr;
    mrow[i] = m < p.M ? m : p.M - 1;
    arow[i] = p.a + mrow[i] * p.lda + 16 * lq;
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int64_t c = n0 + 16 * f + (HALF ? lr & 7 : lr);
    const int64_t n = c < p.N ? c : p.N - 1;
#pragma unroll
    for (int b = 0; b < NP; ++b) brow[b][f] = p.b + ((HALF ? lr >> 3 : b) * p.up + n) * p.ldb + 16 * lq;
  }

  acc_t acc[NP][NF][MF];
#pragma unroll
  for (int b = 0; b < NP; ++b)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < MF; ++i) acc[b][f][i] = acc_t{0, 0, 0, 0};

  const int64_t KG = (p.K + 127) >> 7;            // FP8: K is a multiple of 128
  const int64_t kfull = p.K >> 7;                 // groups wholly inside K

  struct Group {
    Frag a[MF], b[NP][NF];
    float sa[MF], sb[NP];                         // FP8: this group's scales
  };
  auto load = [&](auto tail, Group& x, int64_t g) {
    constexpr bool TAIL = decltype(tail)::value;
    const int64_t left = p.K - 16 * lq;           // K as seen from this lane's first chunk
#pragma unroll
    for (int b = 0; b < NP; ++b)
#pragma unroll
      for (int f = 0; f < NF; ++f) x.b[b][f] = load_frag<TAIL, false>(brow[b][f], g * 128, left);
#pragma unroll
    for (int i = 0; i < MF; ++i) x.a[i] = load_frag<TAIL, TAIL>(arow[i], g * 128, left);
    if constexpr (!INT8) {
#pragma unroll
      for (int i = 0; i < MF; ++i) x.sa[i] = p.sa[g * p.sa_ld + mrow[i]];
#pragma unroll
      for (int b = 0; b < NP; ++b) x.sb[b] = p.sb[(((HALF ? lq >> 1 : b) * p.up + n0) >> 7) * KG + g];
    }
  };
  auto use = [&](const Group& x) {
    if constexpr (INT8) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < NP; ++b)
#pragma unroll
          for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int i = 0; i < MF; ++i)
              acc[b][f][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                  __builtin_bit_cast(v4i, h ? x.b[b][f].hi : x.b[b][f].lo),
                  __builtin_bit_cast(v4i, h ? x.a[i].hi : x.a[i].lo), acc[b][f][i], 0, 0, 0);
    } else {
      const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
      auto v = [](const Frag& f) {
        return v8i{int(f.lo.x), int(f.lo.y), int(f.lo.z), int(f.lo.w), int(f.hi.x), int(f.hi.y), int(f.hi.z), int(f.hi.w)};
      };
#pragma unroll
      for (int b = 0; b < NP; ++b)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int i = 0; i < MF; ++i) {
            const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v(x.b[b][f]), v(x.a[i]), zero, 0, 0, 0, 0, 0, 0);
            const float c = x.sa[i] * x.sb[b];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][f][i][j] = __builtin_fmaf(d[j], c, acc[b][f][i][j]);
          }
    }
  };

  // What the epilogue multiplies and adds is on its way before the weight, one
  // value of each kind per thread (past the end: the last row's or column's).
  const int tid = threadIdx.x;
  float my_sa = 0.0f, my_sb = 0.0f, my_bias = 0.0f;
  if constexpr (INT8) {
    if (p.K > 0 && tid < 16 * MF) my_sa = p.sa[m0 + tid < p.M ? m0 + tid : p.M - 1];
    if (tid < NC * CW) {
      const int64_t c = n0 + tid % CW, n = c < p.N ? c : p.N - 1;
      if (p.K > 0) my_sb = p.sb[tid / CW * p.up + n];
      if (!GATED && p.bias) my_bias = p.bias[n];
    }
  }

  // This wave's contiguous share of the groups: [g, whole) inside K, and up to
  // `end` the group that reaches beyond it.
  int64_t g = KG * wave / WAVES;
  const int64_t end = KG * (wave + 1) / WAVES;
  const int64_t whole = end < kfull ? end : kfull;
  // `n` groups (n <= UNROLL): all loads are issued before the first is used
  auto run = [&](auto full, int n) {
    Group x[UNROLL];
#pragma unroll
    for (int s = 0; s < UNROLL; ++s)
      if (full || s < n) load(std::false_type{}, x[s], g + s);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < UNROLL; ++s)
      if (full || s < n) use(x[s]);
  };
  for (; g + UNROLL <= whole; g += UNROLL) run(std::true_type{}, UNROLL);
  if (g < whole) run(std::false_type{}, int(whole - g));
  if (end > kfull) {
    Group x;
    load(std::true_type{}, x, kfull);
    use(x);
  }

  if constexpr (INT8) {
    if (tid < 16 * MF) s_sa[tid] = my_sa;
    if (tid < NC * CW) {
      s_sb[tid] = my_sb;
      s_bias[tid] = my_bias;
    }
  }
  // The waves' parts meet in LDS, 16 columns at a time.
  const int64_t m = m0 + 16 * wave + lr;
#pragma unroll
  for (int nf = 0; nf < NF; ++nf) {
    if (nf) __syncthreads();
#pragma unroll
    for (int b = 0; b < NP; ++b)
#pragma unroll
      for (int i = 0; i < MF; ++i) part[wave][b * MF + i][lane] = acc[b][nf][i];
    __syncthreads();
    // Wave f adds the parts of row fragment f; a lane finishes four columns of
    // one row (HALF: of lane quarters 0 and 1; the up projection's values are
    // 32 lanes above the gate's).
    if (wave < MF && m < p.M && n0 + 16 * nf + 4 * lq < p.N && (!HALF || lq < 2)) {
      const int64_t n = n0 + 16 * nf + 4 * lq;
      acc_t sum[NC];
#pragma unroll
      for (int b = 0; b < NC; ++b) {
        const int part_b = HALF ? wave : b * MF + wave, part_lane = HALF ? lane + 32 * b : lane;
        sum[b] = part[0][part_b][part_lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum[b] += part[w][part_b][part_lane];
      }
      const int cols = p.N - n < 4 ? int(p.N - n) : 4;
      float y[NC][4], out[4];
#pragma unroll
      for (int b = 0; b < NC; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[b][j] = float(sum[b][j]);
          if constexpr (INT8) y[b][j] *= s_sa[16 * wave + lr] * s_sb[b * CW + 16 * nf + 4 * lq + j];
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (GATED) out[j] = gate_mul(y[0][j], y[1][j], p.act_c1, p.act_c3);
        else out[j] = p.bias ? y[0][j] + s_bias[16 * nf + 4 * lq + j] : y[0][j];
      }
      auto store = [&](void* base, int64_t ld, int64_t col, const float (&v)[4]) {
        if constexpr (OUT == kOutBF16) {
          uint16_t* dst = static_cast<uint16_t*>(base) + m * ld + col;
          const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
          if (cols == 4) {
            *reinterpret_cast<uint2*>(dst) = uint2{lo, hi};
          } else {
            dst[0] = uint16_t(lo);
            if (cols > 1) dst[1] = uint16_t(lo >> 16);
            if (cols > 2) dst[2] = uint16_t(hi);
          }
        } else {
          float* dst = static_cast<float*>(base) + m * ld + col;
          if (cols == 4) {
            *reinterpret_cast<v4f*>(dst) = v4f{v[0], v[1], v[2], v[3]};
          } else {
            dst[0] = v[0];
            if (cols > 1) dst[1] = v[1];
            if (cols > 2) dst[2] = v[2];
          }
        }
      };
      store(p.c, p.ldc, n, out);
      if constexpr (GATED)
        if (p.gu) {
          store(p.gu, p.ldgu, n, y[0]);
          store(p.gu, p.ldgu, p.up + n, y[1]);
        }
    }
  }
}

template <bool INT8, bool GATED, int OUT, int I>
static hipError_t launch_stream_cfg(const FfnArgs& p, hipStream_t st) {
  constexpr StreamKernel S = kStreamKernels[I];
  constexpr int UNROLL = S.mf == 1 && S.nf == 1 ? 4 : 2;
  return in_pieces(p, INT8, OUT == kOutBF16, 16 * S.mf, S.half ? 8 : 16 * S.nf, S.waves * 64,
                   [&](const FfnArgs& q, unsigned grid) {
    hipLaunchKernelGGL((stream_kernel<INT8, GATED, S.half, S.mf, S.nf, S.waves, UNROLL, OUT>), dim3(grid),
                       dim3(S.waves * 64), 0, st, q);
    return hipGetLastError();
  });
}

template <bool INT8, bool GATED, int OUT>
static hipError_t launch_stream(const FfnArgs& p, hipStream_t st) {
  const int i = stream_kernel_for(GATED, p.M, p.N);
  if constexpr (GATED) {
    if (i == 0) return launch_stream_cfg<INT8, GATED, OUT, 0>(p, st);
    if (i == 1) return launch_stream_cfg<INT8, GATED, OUT, 1>(p, st);
  } else {
    if (i == 2) return launch_stream_cfg<INT8, GATED, OUT, 2>(p, st);
    if (i == 3) return launch_stream_cfg<INT8, GATED, OUT, 3>(p, st);
    if (i == 4) return launch_stream_cfg<INT8, GATED, OUT, 4>(p, st);
  }
  switch (i) {
    case 5: return launch_stream_cfg<INT8, GATED, OUT, 5>(p, st);
    case 6: return launch_stream_cfg<INT8, GATED, OUT, 6>(p, st);
    case 7: return launch_stream_cfg<INT8, GATED, OUT, 7>(p, st);
    case 8: return launch_stream_cfg<INT8, GATED, OUT, 8>(p, st);
    default: return launch_stream_cfg<INT8, GATED, OUT, 9>(p, st);
  }
}

}  // namespace fp8q
