// Answers questions about csrc/front/route_choice.h, one a line on standard input:
//   token room E k bits...   ->  near e0 e1 ...   for E FP32 logits, given as integers of their bits, in `room` places
//                                (64 to 1024): whether the kernel would have to choose again, and the k experts that
//                                the keys choose (-1: none left)
#include "front/route_choice.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <functional>
#include <vector>

int main() {
  char what[32];
  int room, experts, k;
  while (std::scanf("%31s %d %d %d", what, &room, &experts, &k) == 4) {
    if (std::strcmp(what, "token") != 0) return 1;
    const uint32_t low = uint32_t(room) - 1u;
    std::vector<uint32_t> sorted;
    std::vector<float> logits;
    for (int e = 0; e < room; ++e) {
      unsigned bits = 0xFF800000u;               // minus infinity beyond the row
      if (e < experts && std::scanf("%u", &bits) != 1) return 1;
      logits.push_back(__builtin_bit_cast(float, uint32_t(bits)));
      sorted.push_back(fp8q::key_of(fp8q::in_order(logits.back()), e, low));
    }
    std::sort(sorted.begin(), sorted.end(), std::greater<uint32_t>());
    uint32_t best[8];
    std::copy_n(sorted.begin(), 8, best);
    bool near = fp8q::close_among<true>(best, low, k);
    if (near && !fp8q::close_among<false>(best, low, k)) return 1;           // which the kernel asks first
    if (k == 8) {
      const float least = fp8q::least_of(best[7], low);
      near |= std::count_if(logits.begin(), logits.end(), [&](float z) { return z >= least; }) > 8;
    }
    std::printf("%d", int(near));
    for (int j = 0; j < k; ++j) std::printf(" %d", best[j] >= fp8q::kLeastKey ? int(low - (best[j] & low)) : -1);
    std::printf("\n");
  }
  return 0;
}
