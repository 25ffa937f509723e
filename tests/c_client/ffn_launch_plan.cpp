// Answers questions about csrc/ffn/launch_plan.h, one a line on standard input:
//   pieces M N bm bn threads   ->  rows cols   of C in one launch
//   kernel gated M N K         ->  the kernels that the product runs in, such as
//                                  "stream 2x1x8", "stream half 1x1x16" (row and column fragments, waves),
//                                  "tile 128x128x2" or "tile 256x256x1 + 64x64x2" (columns split off first)
#include "ffn/launch_plan.h"

#include <cstdio>
#include <cstring>

int main() {
  char what[32];
  while (std::scanf("%31s", what) == 1) {
    long long m, n, k, bm, bn;
    int threads, gated;
    if (std::strcmp(what, "pieces") == 0) {
      if (std::scanf("%lld %lld %lld %lld %d", &m, &n, &bm, &bn, &threads) != 5) return 1;
      const fp8q::Piece p = fp8q::piece_size(m, n, bm, bn, threads);
      std::printf("%lld %lld\n", static_cast<long long>(p.rows), static_cast<long long>(p.cols));
    } else if (std::strcmp(what, "kernel") == 0) {
      if (std::scanf("%d %lld %lld %lld", &gated, &m, &n, &k) != 4) return 1;
      if (fp8q::streams(gated, m, n)) {
        const fp8q::StreamKernel& s = fp8q::kStreamKernels[fp8q::stream_kernel_for(gated, m, n)];
        std::printf("stream %s%dx%dx%d\n", s.half ? "half " : "", s.mf, s.nf, s.waves);
        continue;
      }
      std::printf("tile ");
      for (;;) {
        const fp8q::TilePlan plan = fp8q::tile_plan(gated, m, n, k);
        const fp8q::Tiling& t = fp8q::kTilings[plan.cut ? 0 : plan.tiling];
        std::printf("%dx%dx%d", t.bm, t.bn, t.kw);
        if (!plan.cut) break;
        std::printf(" + ");
        n -= plan.cut;
      }
      std::printf("\n");
    } else {
      return 1;
    }
  }
  return 0;
}
