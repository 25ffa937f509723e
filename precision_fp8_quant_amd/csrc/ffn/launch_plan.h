// Which kernel a gated feed-forward operator's sizes choose, and how its work
// is cut into launches (host only, no HIP).
#pragma once

#include <stdint.h>

namespace fp8q {

// HIP takes launches of fewer than 2^32 threads.
constexpr int64_t max_grid(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

// Workgroups for `units` of them: kernels with a loop over the grid do what is left in further rounds.
inline unsigned grid_of(int64_t units, int threads) {
  return unsigned(units < max_grid(threads) ? units : max_grid(threads));
}

// Rows and columns of C that one launch does of an M x N product in tiles of
// bm x bn, `threads` each.  Launches begin at whole tiles, and at whole 128
// columns, for which FP8 weights have a scale.
struct Piece {
  int64_t rows, cols;
};
inline Piece piece_size(int64_t M, int64_t N, int64_t bm, int64_t bn, int threads) {
  const int64_t most = max_grid(threads), tm = (M - 1) / bm + 1, tn = (N - 1) / bn + 1;
  if (tm <= most / tn) return {M, N};
  const int64_t whole = bn < 128 ? 128 / bn : 1, unit = whole < tn ? whole : tn;
  const int64_t rt = tm < most / unit ? tm : most / unit, ct = most / unit / rt * unit;
  return {rt < tm ? rt * bm : M, ct < tn ? ct * bn : N};
}

// ---- few rows: the weight is streamed (stream_kernel.h) -------------------------

// Whether streaming beats the LDS tiles (tile_kernel.h).  Beyond 16 rows every
// wave fetches as much of A beside its weight again, and streaming takes
// (microseconds per 128-deep K-group and row of B) 3.5e-5 up to 32 rows and
// 5.1e-5, but no less than 0.41 per group, up to 64; the tiles take 0.33 per
// group with few rows of B, 0.44 with 7168, and 3e-5 per row with many.
// Measured (us, streaming / tiles): 32 rows, 7168 rows of B by 18432 36 / 57,
// 36864 by 7168 69 / 63, 4096 by 7168 16 / 17; 64 rows, the same 53 / 64,
// 94 / 67, 23 / 18.5.
inline bool streams(bool gated, int64_t M, int64_t N) {
  const int64_t brows = gated ? 2 * N : N;
  return M <= 16 || (M <= 32 && brows <= 24000) || (M <= 64 && brows > 5500 && brows <= 8600);
}

// A workgroup of `waves` waves owns 16 mf rows x 16 nf columns, or 8 columns
// with gate and up in one fragment (half).
struct StreamKernel {
  bool half;
  int mf, nf, waves;
};
constexpr StreamKernel kStreamKernels[] = {
    {true, 1, 1, 16}, {true, 2, 1, 16},                                        // gated
    {false, 1, 2, 8}, {false, 2, 2, 8}, {false, 4, 2, 8},                      // plain
    {false, 1, 1, 16}, {false, 1, 1, 8}, {false, 2, 1, 16}, {false, 2, 1, 8}, {false, 4, 1, 8}};

// Index of the kernel.  16 waves where there are no more workgroups than CUs
// (FP8 gated 16x2048x7168 by 16 columns 12.2 us a call against 12.5), 8
// otherwise (int8 1x7168x18432 26.0 against 29.8).  Two column fragments per
// wave halve what a plain product fetches of A (int8 16x7168x18432 29.0 against
// 36.8), if they leave enough workgroups; a gated one has its two projections
// already (FP8 16x18432x7168 56.8 with one, 58.9 with two).  Gated with at most
// 2048 columns, up to 32 rows: 8 columns a workgroup, so that a CU streams half
// as much (us with 16 columns / with 8, K = 7168: int8 1x2048 9.8 / 8.6,
// 16x2048 12.0 / 9.2, 32x2048 15.3 / 12.5, 16x512 11.7 / 8.8; FP8 16x2048 12.1 /
// 9.9; with more columns than the CUs hold at once it loses: int8 16x2688 12.1 /
// 16.1).  Eight of a plain product's columns would leave half of each fragment
// empty, and gain nothing.
inline int stream_kernel_for(bool gated, int64_t M, int64_t N) {
  const bool few = (N + 15) / 16 <= 256;
  if (gated && (N + 7) / 8 <= 256 && M <= 32) return M <= 16 ? 0 : 1;
  if (!gated && M > 4 && (N + 31) / 32 >= 192) return M <= 16 ? 2 : M <= 32 ? 3 : 4;
  if (M <= 16) return few ? 5 : 6;
  if (M <= 32) return few ? 7 : 8;
  return 9;
}

// ---- many rows: LDS tiles (tile_kernel.h) ---------------------------------------

// A workgroup computes bm rows by bn rows of B with kw teams of waves that take
// the K-groups in turn; a wave does bm / wm rows by 32 pf rows of B.
struct Tiling {
  int bm, bn, kw, wm, pf;
  float alone, full, tbs, out;    // what the tiling's time is reckoned from, below
};
//   256x256x1  8 waves of 64x128, 1 workgroup per CU
//   128x128x1  4 waves of 64x64, 2
//   128x128x2  8 waves of 64x64, 1
//   64x64x2    8 waves of 16x64, 2
//   64x64x4    16 waves of 16x64, 1
constexpr Tiling kTilings[] = {{256, 256, 1, 4, 4, 1.24f, 1.24f, 2.8f, 7.4f},
                               {128, 128, 1, 2, 2, 0.75f, 0.49f, 3.3f, 3.4f},
                               {128, 128, 2, 2, 2, 0.61f, 0.61f, 2.5f, 2.5f},
                               {64, 64, 2, 4, 2, 0.40f, 0.25f, 2.5f, 1.6f},
                               {64, 64, 4, 4, 2, 0.33f, 0.33f, 2.8f, 1.5f}};

// Microseconds for an M x N product in tiling i.  A larger tile reads fewer
// bytes per product, a smaller one spreads a small problem over more of the 256
// CUs and rounds M and N up less; teams keep a CU busy that has one tile (more
// than two stages do not: a lone 64x64 tile took 35 us for 56 groups with 3 and
// with 6).  Measured microseconds per 128-deep K-group, for a CU's only tile
// (alone), and per tile and CU when the CUs are full (int8, M = 80 .. 4096,
// K = 7168 and 18432; FP8 has the same ratios): the first two columns above.
// A problem runs in rounds.  Where a CU holds one workgroup, each round of 256
// tiles, full or not, takes the one time per group.  Where it holds two, a
// round is 512 tiles and takes twice the second time; a last round takes the
// first time up to 256 tiles and a line between the two beyond.  The time is
// never less than the weight's 128 bytes a row take at the rate that each
// tiling was seen to stream a weight too large for the caches (tbs, TB/s).  To
// this comes what a round takes to fill and to leave (out, us), half of it
// where half a CU's tiles are left.
// The smallest wins.  Measured (us, in the order above):
//   int8  512x7168x7168   70  42  35  48  68
//   int8  128x7168x7168   68  43  35  23  19
//   int8 2048x7168x7168   80  96   -   -   -
//   int8 gated 64x18432x7168   -  67   -  80   -
//   int8 gated 128x18432x7168 94  81 107 107 126
//   FP8 gated 512x2048x7168   80  44  35  26  36
//   FP8 gated 1846x640x6016   70  38  32  41  47   (580 tiles of 64x64)
//   FP8 gated 4096x1408x2048  33  36  43  52  77
//   FP8 gated 2056x14976x640  73  65   - 131   -
//   int8  333x2000x512      10.7 5.8 6.5 4.5 5.1
//   int8 1024x4096x512      11.4 6.9 7.6 9.9 16.7
//   int8 4096x4096x512        15  17  27  35  64
inline float tile_cost(bool gated, int64_t M, int64_t N, int64_t K, int i) {
  const Tiling& s = kTilings[i];
  const int64_t kg = (K + 127) / 128, cn = gated ? s.bn / 2 : s.bn;
  const int64_t tiles = ((M + s.bm - 1) / s.bm) * ((N + cn - 1) / cn), two = s.alone != s.full ? 2 : 1;
  const int64_t last = tiles % (256 * two);
  const float rounds = float(tiles / (256 * two));
  const float beyond = last > 256 ? float(last - 256) / 256.0f : 0.0f;
  const float c = rounds * float(two) * s.full + (last ? s.alone + beyond * (2 * s.full - s.alone) : 0.0f);
  const float stream = float(N * (gated ? 2 : 1)) * 128e-6f / s.tbs;
  const float ends = rounds + (last > 256 || two == 1 ? float(last > 0) : last > 0 ? 0.5f : 0.0f);
  return (c > stream ? c : stream) * float((kg + s.kw - 1) / s.kw * s.kw) + ends * s.out;
}

inline int cheapest_tiling(bool gated, int64_t M, int64_t N, int64_t K) {
  int best = 0;
  for (int i = 1; i < 5; ++i)
    if (tile_cost(gated, M, N, K, i) < tile_cost(gated, M, N, K, best)) best = i;
  return best;
}

// The tiling, and how many leading columns run in 256x256 tiles of their own
// before it: whole columns of such tiles that fill rounds, with the other
// columns right behind them as a problem of their own in smaller tiles, where
// that is less by more than a launch (int8 8192x7168x18432, 3.5 rounds: 857 ->
// 820 us; int8 4200x4096x4096, 272 tiles: 85 -> 70; FP8 gated 2239x4608x3840:
// 100 -> 87).
struct TilePlan {
  int tiling;                     // of all columns where cut is 0; the others are planned on their own otherwise
  int64_t cut;
};
inline TilePlan tile_plan(bool gated, int64_t M, int64_t N, int64_t K) {
  const int best = cheapest_tiling(gated, M, N, K);
  const int64_t cn = gated ? 128 : 256, tm = (M + 255) / 256, tn = (N + cn - 1) / cn;
  const int64_t whole = tm * tn / 256 * 256 / tm, cut = whole * cn;
  if (whole > 0 && whole < tn &&
      tile_cost(gated, M, cut, K, 0) + tile_cost(gated, M, N - cut, K, cheapest_tiling(gated, M, N - cut, K)) + 3.0f <
          tile_cost(gated, M, N, K, best))
    return {best, cut};
  return {best, 0};
}

}  // namespace fp8q
