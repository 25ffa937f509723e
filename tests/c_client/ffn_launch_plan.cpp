// Answers questions about csrc/ffn/launch_plan.h, one a line on standard input:
//   pieces M N bm bn threads   ->  rows cols   of C in one launch
#include "ffn/launch_plan.h"

#include <cstdio>
#include <cstring>

int main() {
  char what[32];
  while (std::scanf("%31s", what) == 1) {
    if (std::strcmp(what, "pieces") != 0) return 1;
    long long m, n, bm, bn;
    int threads;
    if (std::scanf("%lld %lld %lld %lld %d", &m, &n, &bm, &bn, &threads) != 5) return 1;
    const fp8q::Piece p = fp8q::piece_size(m, n, bm, bn, threads);
    std::printf("%lld %lld\n", static_cast<long long>(p.rows), static_cast<long long>(p.cols));
  }
  return 0;
}
