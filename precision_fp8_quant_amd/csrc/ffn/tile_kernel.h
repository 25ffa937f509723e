// Products of 8-bit operands for many rows of A: LDS-tiled, the same operators
// as stream_kernel.h.
//
//   plain:  C[m][n] = sa[m] sb[n] sum_k A[m][k] B[n][k] (+ bias[n])
//   gated:  h[m][f] = act(g) u,  g from B's rows [0, N), u from rows [up, up + N)
//
// The data path is the one of gemm_kernel.h: per 128-deep K-group, global ->
// LDS by LDS DMA (16-byte chunks XOR-swizzled by row, B rows in fragment
// order), ds_read_b128 fragments, matrix instructions issued "swapped" so that
// a lane's results are consecutive columns of one row.  What differs:
//
//  * A wave's columns are two panels of 16 PF columns each (PF fragments).
//    Gated: the gate and the up projection of the same output columns, so the
//    activation and the product happen in the accumulators' own registers and
//    only h leaves the chip (and g, u where the caller keeps them); a tile of
//    BN rows of B gives BN / 2 columns of h.  Plain: two neighbouring panels.
//  * 8-bit integers: the 32-bit sums stay in the matrix instructions'
//    accumulators over the whole of K (two 16x16x64 per 128-deep group), and the
//    scales are applied once, in the epilogue.
//  * Block-scaled FP8: a group's A-row and block scales travel with its stage
//    (4-byte LDS DMA), so nothing in the loop waits on a register load.
//  * KW teams of waves in one workgroup may take a tile's K-groups in turn, each
//    with its own stages; their sums meet in LDS at the end, in a fixed order.
//  * Any M, N (integers) and K (integers): a tile's rows past the end repeat the
//    last valid row (their products are not stored), so every DMA address is
//    inside its operand; in the group that reaches beyond K the A tile's bytes
//    past K are cleared in LDS (0 times any integer is 0).
#pragma once

#include "../gemm_kernel.h"
#include "bf16.h"
#include "ffn_launch.h"
#include "gate_act.h"

namespace fp8q {

typedef int v4i __attribute__((ext_vector_type(4)));

template <bool INT8, bool GATED, int BM, int BN, int WM, int PF, int KW, int OUT>
__global__ __launch_bounds__(KW * WM * (BN / (32 * PF)) * 64) void tile_kernel(FfnArgs p) {
  constexpr int WN = BN / (32 * PF);    // waves along B's rows
  constexpr int NW = WM * WN;           // waves per team; KW teams take the K-groups in turn
  constexpr int TM = BM / WM;           // wave tile rows
  constexpr int SM = TM / 16;           // 16-row subtiles per wave
  constexpr int PC = 16 * PF;           // columns per panel
  constexpr int CN = GATED ? BN / 2 : BN;        // columns of C per tile
  constexpr int A_BYTES = BM * 128;
  constexpr int B_BYTES = BN * 128;
  constexpr int S_BYTES = INT8 ? 0 : BM * 4 + 256;   // FP8: the group's A-row scales, then the two block scales
  constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
  constexpr int A_DMA = A_BYTES / 1024 / NW;     // 1 KB wave-wide DMA instructions per wave per stage
  constexpr int B_DMA = B_BYTES / 1024 / NW;
  static_assert(A_DMA * 1024 * NW == A_BYTES && B_DMA * 1024 * NW == B_BYTES, "DMA split");
  static_assert(INT8 || GATED, "the plain FP8 product is gemm_kernel.h's");
  static_assert(INT8 || (128 % CN == 0 && BM / 64 <= NW), "FP8: a tile in one scale block, one A-scale DMA a wave");
  constexpr int ESZ = OUT == kOutBF16 ? 2 : 4;
  constexpr int PITCH = PC * ESZ + 16;           // bytes per staged output row
  constexpr int LOOP_LDS = KW * 2 * STAGE;
  constexpr int EPI_LDS = NW * TM * PITCH;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LOOP_LDS > EPI_LDS ? LOOP_LDS : EPI_LDS];

  const int lane = threadIdx.x & 63;
  const int team = KW > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / NW : 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) - team * NW;     // within the team
  const int tid = threadIdx.x - team * (NW * 64);
  uint8_t* const smem = lds + team * (2 * STAGE);
  const int wm = wave / WN, wn = wave % WN;
  const int lr = lane & 15, lq = lane >> 4;

  // ---- tile scheduling: every XCD (workgroup i runs on XCD i % 8) gets one
  // contiguous range of tiles, in groups of 8 tiles along M ------------------
  // (The grid has fewer than 2^24 workgroups, so tile numbers are 32-bit.  They
  // are made provably wave-uniform: buffer resources built from values that the
  // compiler holds to be divergent turn every DMA into a loop over the lanes.)
  const uint32_t tiles_m = uint32_t((p.M + BM - 1) / BM);
  const uint32_t tiles_n = uint32_t((p.N + CN - 1) / CN);
  const uint32_t ntiles = tiles_m * tiles_n;
  uint32_t bid = blockIdx.x;
  {
    const uint32_t q = ntiles >> 3, r = ntiles & 7, x = bid & 7, l = bid >> 3;
    bid = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + l;
  }
  constexpr uint32_t GROUP_M = 8;
  const uint32_t per_group = GROUP_M * tiles_n;
  const uint32_t first_m = (bid / per_group) * GROUP_M;
  const uint32_t gsize = (tiles_m - first_m) < GROUP_M ? (tiles_m - first_m) : GROUP_M;
  const int64_t m0 = int64_t(__builtin_amdgcn_readfirstlane(first_m + (bid % per_group) % gsize)) * BM;
  const int64_t n0 = int64_t(__builtin_amdgcn_readfirstlane((bid % per_group) / gsize)) * CN;
  const int mrows = __builtin_amdgcn_readfirstlane(p.M - m0 < BM ? int(p.M - m0) : BM);   // valid rows of A and of
  const int nrows = __builtin_amdgcn_readfirstlane(p.N - n0 < CN ? int(p.N - n0) : CN);   // B (per projection)
  const int64_t KG = (p.K + 127) >> 7;

  // ---- DMA addressing ------------------------------------------------------
  // Wave-wide DMA instruction `blk` fills LDS rows 8*blk .. 8*blk+7; lane l
  // lands at row 8*blk + l/8, physical chunk l%8, i.e. logical chunk
  // (l%8) ^ (l/8).  For B, row 16*js + r of a panel's LDS rows holds the
  // panel's row 4*PF*(r/4) + 4*js + r%4, which leaves every lane with 4*PF
  // consecutive columns.  The byte offset of a lane's row is a constant register
  // per instruction (a clamped row for rows past the end) and the K-group the
  // scalar offset.  Buffer resources end with the last valid row's last 16-byte
  // chunk of K, so the chunks that a last row's final group has beyond K are
  // not read.
  const int lchunk = ((lane & 7) ^ (lane >> 3)) << 4;
  const int kr = int((p.K + 15) & ~int64_t(15));
  const uint8_t* const a_base = p.a + m0 * p.lda;
  const uint8_t* const b_base = p.b + n0 * p.ldb;
  const uint8_t* const u_base = p.b + ((GATED ? p.up : 0) + n0) * p.ldb;
  const int a_end = int((mrows - 1) * p.lda) + kr;
  const int b_end = int((nrows - 1) * p.ldb) + kr;
  int a_off[A_DMA], b_off[B_DMA];
#pragma unroll
  for (int i = 0; i < A_DMA; ++i) {
    const int row = 8 * (wave * A_DMA + i) + (lane >> 3);
    a_off[i] = int((row < mrows ? row : mrows - 1) * p.lda) + lchunk;
  }
#pragma unroll
  for (int i = 0; i < B_DMA; ++i) {
    const int rho = 8 * (wave * B_DMA + i) + (lane >> 3);
    const int panel = rho / PC, js = rho % PC / 16, r = rho % 16;
    const int row = PC * (GATED ? panel >> 1 : panel) + 4 * PF * (r >> 2) + 4 * js + (r & 3);
    b_off[i] = int((row < nrows ? row : nrows - 1) * p.ldb) + lchunk;
  }
  auto issue_dma = [&](int64_t g, int stage, int i) {
    uint8_t* base = smem + stage * STAGE;
    if (i < A_DMA) {
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a_base, (short)0, a_end, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr_t)(base + (wave * A_DMA + i) * 1024), 16, int(a_off[i]),
                                               int(g * 128), 0, 0);
    } else {
      const int blk = wave * B_DMA + i - A_DMA;
      const bool up = GATED && (8 * blk / PC) & 1;
      const __amdgpu_buffer_rsrc_t rsrc =
          __builtin_amdgcn_make_buffer_rsrc((void*)(up ? u_base : b_base), (short)0, b_end, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lptr_t)(base + A_BYTES + blk * 1024), 16, int(b_off[i - A_DMA]),
                                               int(g * 128), 0, 0);
    }
  };
  // FP8: the scales of group g, 4 bytes per lane: 64 A rows by each of the
  // first waves, the gate's and the up's block scale by the last.
  auto issue_scales = [&](int64_t g, int stage) {
    if constexpr (!INT8) {
      uint8_t* const s = smem + stage * STAGE + A_BYTES + B_BYTES;
      if (wave < BM / 64) {
        const int row = 64 * wave + lane;
        const float* src = p.sa + g * p.sa_ld + m0 + (row < mrows ? row : mrows - 1);
        __builtin_amdgcn_global_load_lds((gptr_t)src, (lptr_t)(s + 256 * wave), 4, 0, 0);
      }
      if (wave == NW - 1 && lane < 2) {
        const float* src = p.sb + (((lane ? p.up : 0) + n0) >> 7) * KG + g;
        __builtin_amdgcn_global_load_lds((gptr_t)src, (lptr_t)(s + BM * 4), 4, 0, 0);
      }
    }
  };

  // ---- main loop -------------------------------------------------------------
  typedef typename std::conditional<INT8, v4i, v4f>::type acc_t;
  constexpr int NB = 2 * PF;            // B fragments per group
  constexpr int NT = NB * SM;
  static_assert(A_DMA + B_DMA <= NT, "the next group's DMA rides on this group's first steps");
  acc_t acc[SM][2][PF];
#pragma unroll
  for (int a = 0; a < SM; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int c = 0; c < PF; ++c) acc[a][b][c] = acc_t{0, 0, 0, 0};

  // Team `team` computes groups team, team + KW, ... in two stages of its own
  // (below, "group g" is a team's g-th).  Group 0 is under way before the loop,
  // group g + 1 is requested while group g is computed, into the stage that
  // group g-1 has left.
  // A wave's part of group g has landed once none of its DMAs is outstanding;
  // the barrier then says so for every wave, and that every wave is done with
  // group g-1.  Past the last group the last one is requested again; its copy
  // lands in the stage that is not read any more, before the epilogue's barrier.
  auto clampg = [&](int64_t i) {                  // K-group of this team's i-th turn
    const int64_t g = i * KW + team;
    return g < KG ? g : KG - 1;
  };
  const int64_t turns = (KG + KW - 1) / KW;
  if (KG > 0) {
    issue_scales(clampg(0), 0);
#pragma unroll
    for (int i = 0; i < A_DMA + B_DMA; ++i) issue_dma(clampg(0), 0, i);
  }

  int stage = 0;
  for (int64_t g = 0; g < turns; ++g) {
    wait_vmem_all();
    __syncthreads();
    const int64_t gn = clampg(g + 1);
    const int stage_n = stage ^ 1;
    issue_scales(gn, stage_n);
    uint8_t* const ta = smem + stage * STAGE;
    const uint8_t* const tb = ta + A_BYTES;
    if constexpr (INT8) {
      if (g + 1 == turns && (p.K & 127)) {         // block-uniform
        const int k = int(p.K & 127);
        if (KW == 1 || g * KW + team == KG - 1)
          for (int w = tid; w < BM * 32; w += NW * 64) {         // dword w%32 of row w/32
            const int row = w >> 5, byte = (w & 31) * 4;
            if (byte + 4 > k) {
              uint32_t* dst = reinterpret_cast<uint32_t*>(ta + lds_off(row, byte >> 4) + (byte & 15));
              *dst = byte >= k ? 0u : *dst & ((1u << (8 * (k - byte))) - 1u);
            }
          }
        __syncthreads();
      }
    }
    if (KW > 1 && g * KW + team >= KG) break;      // the last turn has fewer groups than teams; no barrier is left in it

    v8i af[SM];
    v8i bf[3];
#pragma unroll
    for (int ms = 0; ms < SM; ++ms) af[ms] = read_frag(ta, wm * TM + 16 * ms + lr, lq);
    auto frag_row_b = [&](int bi) { return wn * (2 * PC) + 16 * bi + lr; };
    bf[0] = read_frag(tb, frag_row_b(0), lq);
    bf[1] = read_frag(tb, frag_row_b(1), lq);
    if constexpr (INT8) {
      auto half = [](v8i v, int h) { return h ? v4i{v[4], v[5], v[6], v[7]} : v4i{v[0], v[1], v[2], v[3]}; };
#pragma unroll
      for (int bi = 0; bi < NB; ++bi) {
#pragma unroll
        for (int s = 0; s < 2 * SM; ++s) {         // the two halves of K in turn over all rows: no back-to-back dependence
          const int ms = s % SM;
          acc[ms][bi / PF][bi % PF] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              half(bf[bi % 3], s / SM), half(af[ms], s / SM), acc[ms][bi / PF][bi % PF], 0, 0, 0);
          if (s == 0 && bi + 2 < NB) bf[(bi + 2) % 3] = read_frag(tb, frag_row_b(bi + 2), lq);
          const int t = bi * 2 * SM + s;
          if (t % 2 == 0 && t / 2 < A_DMA + B_DMA) issue_dma(gn, stage_n, t / 2);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
      const float* const sc = reinterpret_cast<const float*>(tb + B_BYTES);
      float cs[2][SM];                             // combined scale per projection and row
      const float sg = sc[BM], su = sc[BM + 1];
#pragma unroll
      for (int ms = 0; ms < SM; ++ms) {
        const float sa = sc[wm * TM + 16 * ms + lr];
        cs[0][ms] = sa * sg;
        cs[1][ms] = sa * su;
      }
      v4f dq[3];
      const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < NT + 2; ++t) {           // step t's matrix instruction, then step t-2's promotion
        if (t < NT) {
          const int bi = t / SM, ms = t % SM;
          dq[t % 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[bi % 3], af[ms], zero, 0, 0, 0, 0, 0, 0);
          if (ms == 0 && bi + 2 < NB) bf[(bi + 2) % 3] = read_frag(tb, frag_row_b(bi + 2), lq);
          if (t < A_DMA + B_DMA) issue_dma(gn, stage_n, t);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (t >= 2) {
          const int bu = (t - 2) / SM, mu = (t - 2) % SM;
          const v4f d = dq[(t - 2) % 3];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[mu][bu / PF][bu % PF][j] = __builtin_fmaf(d[j], cs[bu / PF][mu], acc[mu][bu / PF][bu % PF][j]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    stage ^= 1;
  }
  wait_vmem_all();                               // what follows reuses the stages
  __syncthreads();

  // The teams' sums meet in the first one's registers, in the teams' order.
  if constexpr (KW > 1) {
    constexpr int FR = SM * 2 * PF;
    static_assert((KW - 1) * NW * FR * 1024 <= int(sizeof(lds)), "the teams' sums fit the stages");
    acc_t* const red = reinterpret_cast<acc_t*>(lds) + lane;
    if (team > 0) {
#pragma unroll
      for (int i = 0; i < FR; ++i)
        red[(((team - 1) * NW + wave) * FR + i) * 64] = acc[i / (2 * PF)][i / PF % 2][i % PF];
    }
    __syncthreads();
    if (team == 0) {
#pragma unroll
      for (int k = 0; k < KW - 1; ++k)
#pragma unroll
        for (int i = 0; i < FR; ++i) acc[i / (2 * PF)][i / PF % 2][i % PF] += red[((k * NW + wave) * FR + i) * 64];
    }
    __syncthreads();                             // the output tile is staged over the sums
    if (team > 0) return;
  }

  // ---- epilogue --------------------------------------------------------------
  // As in gemm_kernel.h the tile leaves through LDS, one panel per wave at a
  // time, so that a store instruction writes whole runs of a row.
  const int64_t n_wave = n0 + wn * (GATED ? PC : 2 * PC);
  float y[SM][2][PF][4];
#pragma unroll
  for (int ms = 0; ms < SM; ++ms)
#pragma unroll
    for (int pn = 0; pn < 2; ++pn)
#pragma unroll
      for (int js = 0; js < PF; ++js)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[ms][pn][js][j] = float(acc[ms][pn][js][j]);
  if constexpr (INT8) {
    if (KG > 0) {
      float sa[SM];
#pragma unroll
      for (int ms = 0; ms < SM; ++ms) {
        const int64_t m = m0 + wm * TM + 16 * ms + lr;
        sa[ms] = p.sa[m < p.M ? m : p.M - 1];
      }
#pragma unroll
      for (int pn = 0; pn < 2; ++pn)
#pragma unroll
        for (int js = 0; js < PF; ++js)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t c = n_wave + (GATED ? 0 : PC * pn) + 4 * PF * lq + 4 * js + j;
            const float sb = p.sb[(GATED && pn ? p.up : 0) + (c < p.N ? c : p.N - 1)];
#pragma unroll
            for (int ms = 0; ms < SM; ++ms) y[ms][pn][js][j] *= sa[ms] * sb;
          }
    }
    if constexpr (!GATED) {
      if (p.bias) {
#pragma unroll
        for (int pn = 0; pn < 2; ++pn)
#pragma unroll
          for (int js = 0; js < PF; ++js)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int64_t c = n_wave + PC * pn + 4 * PF * lq + 4 * js + j;
              const float b = p.bias[c < p.N ? c : p.N - 1];
#pragma unroll
              for (int ms = 0; ms < SM; ++ms) y[ms][pn][js][j] += b;
            }
      }
    }
  }

  constexpr int LPR = PC * ESZ / 16;             // lanes per panel row
  constexpr int RPI = 64 / LPR;                  // rows per store instruction
  constexpr int EPC = 16 / ESZ;                  // elements per 16-byte chunk
  uint8_t* const stg = smem + wave * (TM * PITCH);
  // panel pn of y -> columns [col0, col0 + PC) of dst, columns valid below `end`
  auto emit = [&](int pn, void* dst, int64_t ld, int64_t col0, int64_t end) {
#pragma unroll
    for (int ms = 0; ms < SM; ++ms) {
      uint8_t* row = stg + (16 * ms + lr) * PITCH + 4 * PF * ESZ * lq;
#pragma unroll
      for (int js = 0; js < PF; ++js) {
        const float(&v)[4] = y[ms][pn][js];
        if constexpr (OUT == kOutBF16)
          *reinterpret_cast<uint2*>(row + 8 * js) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        else
          *reinterpret_cast<v4f*>(row + 16 * js) = v4f{v[0], v[1], v[2], v[3]};
      }
    }
    const int chunk = lane % LPR;
    const int64_t n = col0 + chunk * EPC;
    // BF16 rows of whole 128-byte lines go past the caches (int8 8192x7168x18432
    // 824 us, 832 kept in them); others leave partial lines that the L2 has to
    // join first (2000x9300x1024 BF16 48.8 us past the caches, 33.0 through
    // them; FP32 66.6 and 40.8), and FP32 gains from them anyhow (2048x8192x1024
    // 27.2 and 25.3).
    const bool past_cache =
        ESZ == 2 && ((ld * ESZ | int64_t(reinterpret_cast<uintptr_t>(dst)) | col0 * ESZ) & 127) == 0;
#pragma unroll
    for (int sr = 0; sr < (TM + RPI - 1) / RPI; ++sr) {
      const int r = sr * RPI + lane / LPR;
      const int64_t m = m0 + wm * TM + r;
      if ((TM % RPI && r >= TM) || m >= p.M || n >= end) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(stg + r * PITCH + 16 * chunk);
      uint8_t* out = static_cast<uint8_t*>(dst) + (m * ld + n) * ESZ;
      if (n + EPC <= end) {
        if (past_cache) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(out));
        else *reinterpret_cast<u32x4*>(out) = v;
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
      emit(1, p.gu, p.ldgu, p.up + n_wave, p.up + p.N);
    }
#pragma unroll
    for (int ms = 0; ms < SM; ++ms)
#pragma unroll
      for (int js = 0; js < PF; ++js)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[ms][0][js][j] = gate_mul(y[ms][0][js][j], y[ms][1][js][j], p.act_c1, p.act_c3);
    emit(0, p.c, p.ldc, n_wave, p.N);
  } else {
    emit(0, p.c, p.ldc, n_wave, p.N);
    emit(1, p.c, p.ldc, n_wave + PC, p.N);
  }
}

template <bool INT8, bool GATED, int OUT, int I>
static hipError_t launch_tile_cfg(const FfnArgs& p, hipStream_t st) {
  constexpr Tiling T = kTilings[I];
  constexpr int THREADS = T.kw * T.wm * (T.bn / (32 * T.pf)) * 64;
  return in_pieces(p, INT8, OUT == kOutBF16, T.bm, GATED ? T.bn / 2 : T.bn, THREADS, [&](const FfnArgs& q, unsigned grid) {
    hipLaunchKernelGGL((tile_kernel<INT8, GATED, T.bm, T.bn, T.wm, T.pf, T.kw, OUT>), dim3(grid), dim3(THREADS), 0, st, q);
    return hipGetLastError();
  });
}

template <bool INT8, bool GATED, int OUT>
static hipError_t launch_tile(const FfnArgs& p, hipStream_t st) {
  const TilePlan plan = tile_plan(GATED, p.M, p.N, p.K);
  if (plan.cut) {
    const FfnArgs head = part_of(p, INT8, OUT == kOutBF16, 0, p.M, 0, plan.cut);
    const FfnArgs rest = part_of(p, INT8, OUT == kOutBF16, 0, p.M, plan.cut, p.N - plan.cut);
    const hipError_t e = launch_tile_cfg<INT8, GATED, OUT, 0>(head, st);
    return e != hipSuccess ? e : launch_tile<INT8, GATED, OUT>(rest, st);
  }
  switch (plan.tiling) {
    case 0: return launch_tile_cfg<INT8, GATED, OUT, 0>(p, st);
    case 1: return launch_tile_cfg<INT8, GATED, OUT, 1>(p, st);
    case 2: return launch_tile_cfg<INT8, GATED, OUT, 2>(p, st);
    case 3: return launch_tile_cfg<INT8, GATED, OUT, 3>(p, st);
    default: return launch_tile_cfg<INT8, GATED, OUT, 4>(p, st);
  }
}

}  // namespace fp8q
