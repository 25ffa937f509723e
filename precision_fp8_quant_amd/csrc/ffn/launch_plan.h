// How the work of a gated feed-forward operator is cut into launches, as
// functions of its sizes (host only, no HIP).
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

}  // namespace fp8q
