// Keys of the merged choice: a logit's upper bits in the order of the logits,
// and below them the expert, whose complement in `low` (all bits that hold it)
// puts lower indexes first.  Plain C++, for the kernel and for the host.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define FP8Q_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FP8Q_HOST_DEVICE inline
#endif

namespace fp8q {

// Integer of the same order as v; both zeros are the same.
FP8Q_HOST_DEVICE uint32_t in_order(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

// A key below this is that of minus infinity (or of no number).
constexpr uint32_t kLeastKey = 0x00800000u;

// o: the logit as an integer of its order
FP8Q_HOST_DEVICE uint32_t key_of(uint32_t o, int expert, uint32_t low) { return (o & ~low) | (low - uint32_t(expert)); }

// The bits that the keys leave out might order a token's k first choices, 4 <= k
// <= 8, otherwise where one of them holds the same bits of its logit as the next
// key.  Equal bits are neighbours, so behind the k-th only the next matters, and
// keys of minus infinity are no choice.  (65536 tokens of FP32 logits in a graph,
// us, so / with any two of the eight, k or not, counted and keys of minus infinity
// too: 4 of 6 experts 13.3 / 18.0, 7 of 7 13.8 / 19.4, 8 of 64 with nine tenths
// masked 15.4 / 20.6, 4 of 256 28.3 / 32.1, 8 of 64 15.5 / 15.3.)
//
// Among the eight largest keys in descending order.  Without LIVE those of minus
// infinity count, which is quicker to tell (8 of 512 54.1, alone with it 55.8).
template <bool LIVE>
FP8Q_HOST_DEVICE bool close_among(const uint32_t (&best)[8], uint32_t low, int k) {
  uint32_t gap = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < k && (!LIVE || best[j] >= kLeastKey)) {
      const uint32_t d = best[j] ^ best[j + 1];    // no two keys are equal
      gap = d < gap ? d : gap;
    }
  return gap <= low;
}
// The eighth and what is behind it: more than eight of the token's logits are at
// least this, the least one with the eighth key's bits (no number, which none is
// at least, for the key of minus infinity).
FP8Q_HOST_DEVICE float least_of(uint32_t key, uint32_t low) {
  const uint32_t o = key & ~low;
  return __builtin_bit_cast(float, int32_t(o) < 0 ? o ^ 0x80000000u : ~o);
}

}  // namespace fp8q
