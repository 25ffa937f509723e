// Products of 8-bit operands for many rows of A: LDS-tiled, the same operators
// as stream_kernel.h.
//
//   plain:  C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k] (+ bias[n])
//   gated:  h[m][f] = act(g) u,  g from B's rows [0, N), u from rows [N, 2N)
//
// The data path is the one of gemm_kernel.h: per 128-deep K-group, global ->
// LDS by LDS DMA one group ahead into the other of two stages (16-byte chunks
// XOR-swizzled by row, B rows in fragment order), ds_read_b128 fragments, matrix
// instructions issued "swapped" so that a lane's results are 16 consecutive
// columns of one row per 64-column panel.  What differs:
//
//  * Gated: a wave's two 64-column panels are the gate and the up projection of
//    the same 64 output columns, so the activation and the product happen in
//    the accumulators' own registers and only h leaves the chip (and g, u where
//    the caller keeps them).  A tile of BN rows of B gives BN / 2 columns of h.
//  * 8-bit integers: the 32-bit sums stay in the matrix instructions'
//    accumulators over the whole of K (two 16x16x64 per 128-deep group), and the
//    scales are applied once, in the epilogue.
//  * Any M, N (integers) and K (integers): a tile's rows past the end repeat the
//    last valid row (their products are not stored), so every DMA address is
//    inside its operand; in the group that reaches beyond K the A tile's bytes
//    past K are cleared in LDS (0 times any integer is 0).
#pragma once

#include "../gemm_kernel.h"
#include "ffn_launch.h"
#include "gate_act.h"

namespace fp8q {

typedef int v4i __attribute__((ext_vector_type(4)));

template <bool INT8, bool GATED, int BM, int BN, int WM, int OUT>
__global__ __launch_bounds__(WM * (BN / 128) * 64) void tile_kernel(FfnArgs p) {
  constexpr int WN = BN / 128;          // waves along B's rows, 128 each
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM;           // wave tile rows
  constexpr int SM = TM / 16;           // 16-row subtiles per wave
  constexpr int CN = GATED ? BN / 2 : BN;        // columns of C per tile
  constexpr int A_BYTES = BM * 128;
  constexpr int B_BYTES = BN * 128;
  constexpr int STAGE = A_BYTES + B_BYTES;
  constexpr int A_DMA = A_BYTES / 1024 / NW;     // 1 KB wave-wide DMA instructions per wave per stage
  constexpr int B_DMA = B_BYTES / 1024 / NW;
  static_assert(A_DMA * 1024 * NW == A_BYTES && B_DMA * 1024 * NW == B_BYTES, "DMA split");
  static_assert(INT8 || GATED, "the plain FP8 product is gemm_kernel.h's");
  constexpr int ESZ = OUT == kOutBF16 ? 2 : 4;
  constexpr int PITCH = 64 * ESZ + 16;           // bytes per staged output row
  constexpr int LOOP_LDS = 2 * STAGE;
  constexpr int EPI_LDS = NW * TM * PITCH;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LOOP_LDS > EPI_LDS ? LOOP_LDS : EPI_LDS];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int lr = lane & 15, lq = lane >> 4;

  // ---- tile scheduling: every XCD (workgroup i runs on XCD i % 8) gets one
  // contiguous range of tiles, in groups of 8 tiles along M ------------------
  const int64_t tiles_m = (p.M + BM - 1) / BM;
  const int64_t tiles_n = (p.N + CN - 1) / CN;
  const int64_t ntiles = tiles_m * tiles_n;
  int64_t bid = blockIdx.x;
  {
    const int64_t q = ntiles >> 3, r = ntiles & 7, x = bid & 7, l = bid >> 3;
    bid = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + l;
  }
  constexpr int64_t GROUP_M = 8;
  const int64_t per_group = GROUP_M * tiles_n;
  const int64_t first_m = (bid / per_group) * GROUP_M;
  const int64_t gsize = (tiles_m - first_m) < GROUP_M ? (tiles_m - first_m) : GROUP_M;
  const int64_t m0 = (first_m + (bid % per_group) % gsize) * BM;
  const int64_t n0 = ((bid % per_group) / gsize) * CN;
  const int mrows = p.M - m0 < BM ? int(p.M - m0) : BM;        // valid rows of A and of B (per projection)
  const int nrows = p.N - n0 < CN ? int(p.N - n0) : CN;

  // ---- DMA addressing ------------------------------------------------------
  // Wave-wide DMA instruction `blk` fills LDS rows 8*blk .. 8*blk+7; lane l
  // lands at row 8*blk + l/8, physical chunk l%8, i.e. logical chunk
  // (l%8) ^ (l/8).  For B, LDS row rho of panel rho/64 holds the row
  // 16*(r/4) + 4*js + r%4 (rho%64 = 16*js + r) of that panel's 64.  The byte
  // offset of a lane's row is a constant register per instruction (a clamped
  // row for rows past the end) and the K-group the scalar offset.  Buffer
  // resources end with the last valid row's last 16-byte chunk of K, so the
  // chunks that a last row's final group has beyond K are not read.
  const int lchunk = ((lane & 7) ^ (lane >> 3)) << 4;
  const int kr = int((p.K + 15) & ~int64_t(15));
  const __amdgpu_buffer_rsrc_t rsrc_a = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.a + m0 * p.lda), (short)0, int((mrows - 1) * p.lda + kr), 0x00020000);
  // gated: a wave's share of B lies in one panel, the gate's or the up's
  static_assert(!GATED || 8 % B_DMA == 0, "a wave's B share lies in one panel");
  const int64_t b_row0 = n0 + (GATED && ((wave * B_DMA) >> 3 & 1) ? p.N : 0);
  const __amdgpu_buffer_rsrc_t rsrc_b = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(p.b + b_row0 * p.ldb), (short)0, int((nrows - 1) * p.ldb + kr), 0x00020000);
  int a_off[A_DMA], b_off[B_DMA];
#pragma unroll
  for (int i = 0; i < A_DMA; ++i) {
    const int row = 8 * (wave * A_DMA + i) + (lane >> 3);
    a_off[i] = int((row < mrows ? row : mrows - 1) * p.lda) + lchunk;
  }
#pragma unroll
  for (int i = 0; i < B_DMA; ++i) {
    const int blk = wave * B_DMA + i;
    const int panel = GATED ? blk >> 4 : blk >> 3;
    const int row = 64 * panel + 32 * (blk & 1) + 4 * ((blk >> 1) & 3) + 16 * (lane >> 5) + ((lane >> 3) & 3);
    b_off[i] = int((row < nrows ? row : nrows - 1) * p.ldb) + lchunk;
  }
  auto issue_dma = [&](int64_t g, int stage, int i) {
    uint8_t* base = smem + stage * STAGE;
    if (i < A_DMA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_a, (lptr_t)(base + (wave * A_DMA + i) * 1024), 16,
                                               int(a_off[i]), int(g * 128), 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_b,
                                               (lptr_t)(base + A_BYTES + (wave * B_DMA + i - A_DMA) * 1024), 16,
                                               int(b_off[i - A_DMA]), int(g * 128), 0, 0);
  };

  // ---- main loop -------------------------------------------------------------
  typedef typename std::conditional<INT8, v4i, v4f>::type acc_t;
  constexpr int NB = 8;                 // B fragments per group: 2 panels x 4 subtiles
  constexpr int NT = NB * SM;
  static_assert(A_DMA + B_DMA <= NT, "the next group's DMA rides on this group's first steps");
  acc_t acc[SM][2][4];
#pragma unroll
  for (int a = 0; a < SM; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[a][b][c] = acc_t{0, 0, 0, 0};

  const int64_t KG = (p.K + 127) >> 7;
  int64_t m_lane[SM];                   // rows past the end repeat the last one
#pragma unroll
  for (int ms = 0; ms < SM; ++ms) {
    const int64_t m = m0 + wm * TM + 16 * ms + lr;
    m_lane[ms] = m < p.M ? m : p.M - 1;
  }
  const int64_t n_wave = n0 + wn * (GATED ? 64 : 128);
  const float* const sbg = p.sb + (n_wave >> 7) * KG;                  // FP8: gate and up block scales
  const float* const sbu = p.sb + ((p.N + n_wave) >> 7) * KG;
  float sa_cur[SM], sa_nxt[SM], sb_cur[2], sb_nxt[2];
  auto load_scales = [&](int64_t g, float (&sa)[SM], float (&sb)[2]) {
    if constexpr (!INT8) {
#pragma unroll
      for (int ms = 0; ms < SM; ++ms) sa[ms] = p.sa[g * p.M + m_lane[ms]];
      sb[0] = sbg[g];
      sb[1] = sbu[g];
    }
  };
  if (KG > 0) {
#pragma unroll
    for (int i = 0; i < A_DMA + B_DMA; ++i) issue_dma(0, 0, i);
    load_scales(0, sa_cur, sb_cur);
    wait_vmem_all();
  }
  __syncthreads();

  for (int64_t g = 0; g < KG; ++g) {
    const int stage = int(g & 1);
    const int64_t gn = g + 1 < KG ? g + 1 : g;     // the last iteration re-fetches its own group into the idle stage
    uint8_t* const ta = smem + stage * STAGE;
    const uint8_t* const tb = ta + A_BYTES;
    if constexpr (INT8) {
      if (g + 1 == KG && (p.K & 127)) {            // block-uniform
        const int k = int(p.K & 127);
        for (int w = tid; w < BM * 32; w += NW * 64) {           // dword w%32 of row w/32
          const int row = w >> 5, byte = (w & 31) * 4;
          if (byte + 4 > k) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(ta + lds_off(row, byte >> 4) + (byte & 15));
            *dst = byte >= k ? 0u : *dst & ((1u << (8 * (k - byte))) - 1u);
          }
        }
        __syncthreads();
      }
    }
    load_scales(gn, sa_nxt, sb_nxt);

    v8i af[SM];
    v8i bf[3];
#pragma unroll
    for (int ms = 0; ms < SM; ++ms) af[ms] = read_frag(ta, wm * TM + 16 * ms + lr, lq);
    auto frag_row_b = [&](int bi) { return wn * 128 + 16 * bi + lr; };
    bf[0] = read_frag(tb, frag_row_b(0), lq);
    bf[1] = read_frag(tb, frag_row_b(1), lq);
    if constexpr (INT8) {
      auto half = [](v8i v, int h) { return h ? v4i{v[4], v[5], v[6], v[7]} : v4i{v[0], v[1], v[2], v[3]}; };
#pragma unroll
      for (int bi = 0; bi < NB; ++bi) {
#pragma unroll
        for (int s = 0; s < 2 * SM; ++s) {         // the two halves of K in turn over all rows: no back-to-back dependence
          const int ms = s % SM;
          acc[ms][bi >> 2][bi & 3] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              half(bf[bi % 3], s / SM), half(af[ms], s / SM), acc[ms][bi >> 2][bi & 3], 0, 0, 0);
          if (s == 0 && bi + 2 < NB) bf[(bi + 2) % 3] = read_frag(tb, frag_row_b(bi + 2), lq);
          const int t = bi * 2 * SM + s;
          if (t % 2 == 0 && t / 2 < A_DMA + B_DMA) issue_dma(gn, stage ^ 1, t / 2);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
      float cs[2][SM];                             // combined scale per projection and row
#pragma unroll
      for (int ms = 0; ms < SM; ++ms) {
        cs[0][ms] = sa_cur[ms] * sb_cur[0];
        cs[1][ms] = sa_cur[ms] * sb_cur[1];
      }
      v4f dq[3];
      const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < NT + 2; ++t) {           // step t's matrix instruction, then step t-2's promotion
        if (t < NT) {
          const int bi = t / SM, ms = t % SM;
          dq[t % 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[bi % 3], af[ms], zero, 0, 0, 0, 0, 0, 0);
          if (ms == 0 && bi + 2 < NB) bf[(bi + 2) % 3] = read_frag(tb, frag_row_b(bi + 2), lq);
          if (t < A_DMA + B_DMA) issue_dma(gn, stage ^ 1, t);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (t >= 2) {
          const int bu = (t - 2) / SM, mu = (t - 2) % SM;
          const v4f d = dq[(t - 2) % 3];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[mu][bu >> 2][bu & 3][j] = __builtin_fmaf(d[j], cs[bu >> 2][mu], acc[mu][bu >> 2][bu & 3][j]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int ms = 0; ms < SM; ++ms) sa_cur[ms] = sa_nxt[ms];
      sb_cur[0] = sb_nxt[0];
      sb_cur[1] = sb_nxt[1];
    }
    wait_vmem_all();
    __syncthreads();
  }

  // ---- epilogue --------------------------------------------------------------
  // As in gemm_kernel.h the tile leaves through LDS, one 64-column panel per
  // wave at a time, so that every store instruction writes whole lines.
  float y[SM][2][4][4];
#pragma unroll
  for (int ms = 0; ms < SM; ++ms)
#pragma unroll
    for (int pn = 0; pn < 2; ++pn)
#pragma unroll
      for (int js = 0; js < 4; ++js)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[ms][pn][js][j] = float(acc[ms][pn][js][j]);
  if constexpr (INT8) {
    if (KG > 0) {
      float sa[SM];
#pragma unroll
      for (int ms = 0; ms < SM; ++ms) sa[ms] = p.sa[m_lane[ms]];
#pragma unroll
      for (int pn = 0; pn < 2; ++pn)
#pragma unroll
        for (int js = 0; js < 4; ++js)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t c = n_wave + (GATED ? 0 : 64 * pn) + 16 * lq + 4 * js + j;
            const float sb = p.sb[(GATED && pn ? p.N : 0) + (c < p.N ? c : p.N - 1)];
#pragma unroll
            for (int ms = 0; ms < SM; ++ms) y[ms][pn][js][j] *= sa[ms] * sb;
          }
    }
    if constexpr (!GATED) {
      if (p.bias) {
#pragma unroll
        for (int pn = 0; pn < 2; ++pn)
#pragma unroll
          for (int js = 0; js < 4; ++js)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t c = n_wave + 64 * pn + 16 * lq + 4 * js + j;
              const float b = p.bias[c < p.N ? c : p.N - 1];
#pragma unroll
              for (int ms = 0; ms < SM; ++ms) y[ms][pn][js][j] += b;
            }
      }
    }
  }

  constexpr int LPR = 64 * ESZ / 16;             // lanes per 64-column row
  constexpr int RPI = 64 / LPR;                  // rows per store instruction
  constexpr int EPC = 16 / ESZ;                  // elements per 16-byte chunk
  uint8_t* const stg = smem + wave * (TM * PITCH);
  // panel pn of y -> columns [col0, col0 + 64) of dst, columns valid below `end`
  auto emit = [&](int pn, void* dst, int64_t ld, int64_t col0, int64_t end) {
#pragma unroll
    for (int ms = 0; ms < SM; ++ms) {
      uint8_t* row = stg + (16 * ms + lr) * PITCH;
      if constexpr (OUT == kOutBF16) {
        uint32_t w[8];
#pragma unroll
        for (int js = 0; js < 4; ++js) {
          w[2 * js] = bf16_rne_bits(y[ms][pn][js][0]) | (bf16_rne_bits(y[ms][pn][js][1]) << 16);
          w[2 * js + 1] = bf16_rne_bits(y[ms][pn][js][2]) | (bf16_rne_bits(y[ms][pn][js][3]) << 16);
        }
        *reinterpret_cast<u32x4*>(row + 32 * lq) = u32x4{w[0], w[1], w[2], w[3]};
        *reinterpret_cast<u32x4*>(row + 32 * lq + 16) = u32x4{w[4], w[5], w[6], w[7]};
      } else {
#pragma unroll
        for (int js = 0; js < 4; ++js)
          *reinterpret_cast<v4f*>(row + 64 * lq + 16 * js) =
              v4f{y[ms][pn][js][0], y[ms][pn][js][1], y[ms][pn][js][2], y[ms][pn][js][3]};
      }
    }
    const int chunk = lane % LPR;
    const int64_t n = col0 + chunk * EPC;
#pragma unroll
    for (int sr = 0; sr < TM / RPI; ++sr) {
      const int r = sr * RPI + lane / LPR;
      const u32x4 v = *reinterpret_cast<const u32x4*>(stg + r * PITCH + 16 * chunk);
      const int64_t m = m0 + wm * TM + r;
      if (m >= p.M || n >= end) continue;
      uint8_t* out = static_cast<uint8_t*>(dst) + (m * ld + n) * ESZ;
      if (n + EPC <= end) {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out));
      } else {
        for (int e = 0; e < int(end - n); ++e) {
          if constexpr (OUT == kOutBF16)
            reinterpret_cast<uint16_t*>(out)[e] = uint16_t(e & 1 ? v[e >> 1] >> 16 : v[e >> 1]);
          else
            reinterpret_cast<uint32_t*>(out)[e] = v[e];
        }
      }
    }
  };
  if constexpr (GATED) {
    if (p.gu) {
      emit(0, p.gu, p.ldgu, n_wave, p.N);
      emit(1, p.gu, p.ldgu, p.N + n_wave, 2 * p.N);
    }
#pragma unroll
    for (int ms = 0; ms < SM; ++ms)
#pragma unroll
      for (int js = 0; js < 4; ++js)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[ms][0][js][j] = gate_mul(y[ms][0][js][j], y[ms][1][js][j], p.act_c1, p.act_c3);
    emit(0, p.c, p.ldc, n_wave, p.N);
  } else {
    emit(0, p.c, p.ldc, n_wave, p.N);
    emit(1, p.c, p.ldc, n_wave + 64, p.N);
  }
}

template <bool INT8, bool GATED, int BM, int BN, int WM, int OUT>
static hipError_t launch_tile_cfg(const FfnArgs& p, hipStream_t st) {
  constexpr int CN = GATED ? BN / 2 : BN;
  const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + CN - 1) / CN);
  hipLaunchKernelGGL((tile_kernel<INT8, GATED, BM, BN, WM, OUT>), dim3(unsigned(tiles)), dim3(WM * (BN / 128) * 64),
                     0, st, p);
  return hipGetLastError();
}

template <bool INT8, bool GATED, int OUT>
static hipError_t launch_tile(const FfnArgs& p, hipStream_t st) {
  if (p.M > 128) return launch_tile_cfg<INT8, GATED, 256, 256, 4, OUT>(p, st);
  return launch_tile_cfg<INT8, GATED, 128, 256, 2, OUT>(p, st);
}

}  // namespace fp8q
