// The k experts of each token, their weights, the tokens of each expert and the
// loss that balances them; and the gradient with respect to the logits.
//
//   p = softmax(z);  loss = sum_e slope_e sum_t p_te,  slope_e = E c_e / (k n^2)
//   dz = p (dp - sum p dp),  dp_e = dloss slope_e + [e chosen] dc
// LPT lanes share a token and hold its logits in registers, C runs of 8 each
// (expert (c LPT + lane) 8 + j): one read of the logits serves the softmax and
// the choice.  The choice goes by the logits themselves, as integers of the same
// order, so that equal logits are equal, and lower indexes go first:
//   4 to 8 experts  keys of a logit and its expert in one integer; every lane sorts
//                   its runs, and the eights of lanes are merged, level by level.
//                   BF16 leaves 16 bits for the expert.  FP32 loses 6 to 10 of its
//                   bits, and where this could matter to the choice (route_choice.h;
//                   8 of normal logits: one of 4200 tokens of 64, one of 500 of 256)
//                   the wave chooses again by
//   any number      rounds: every lane sorts its runs with all their bits, each of
//                   the k rounds takes the largest of their heads over the lanes and
//                   moves that run up.
// (65536 tokens, merged / by rounds, us: 8 of 64 BF16 9.7 / 11.9, FP32 11.9 / 13.7,
// 8 of 256 FP32 26.3 / 32.5, 8 of 1000 (16384) 31.1 / 34.8, 4 of 64 BF16 9.1 / 9.6;
// 2 of 64 a call 12.5 / 12.1, 2 of 1000 34.1 / 31.7.  16 of 64 BF16 by rounds 13.8,
// 16 of 256 FP32 40.7.)
//
// A lane has the same 8 C experts in all of its workgroup's tokens and sums
// their p in registers, a wave its groups', a workgroup its waves'; workgroups
// leave one row of sums and counts each, which a second kernel adds in a fixed
// order.  With one workgroup it is all one launch.
// Bound by the vector units, which issue for 5.2 us of the 9.7 (8 of 64 BF16; 6 us
// are without the choice), 17.4 of 26.3 (8 of 256 FP32) and 35.5 of 40.7 (16 of 256
// by rounds), and by a launch's start and end and the loads of a turn, that nothing
// hides; then 3.9 us for the sums.  The gradient is bound by memory: 8 of 256 FP32
// 27.5 us a call, 5.0 TB/s, 8 of 1000 (16384 tokens) 26.5, 5.0; BF16 with fewer
// experts by both (8 of 64, 65536 tokens, 8.1 us a call, 4.4 of them vector
// instructions; 8 of 128 11.0 and 8.0).
#include "front_launch.h"
#include "lanes.h"
#include "route_choice.h"
#include "row_io.h"

#include <type_traits>

namespace fp8q {
namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr uint32_t kNegInf = 0xFF800000u;

// A lane's logits of one token as they lie in memory.
template <typename T, int LPT, int C>
struct Logits {
  Row8<T> raw[C];
  __device__ __forceinline__ void load(const T* row, int lane, int cols) {
#pragma unroll
    for (int c = 0; c < C; ++c) load_raw(raw[c], row, (c * LPT + lane) * 8, cols);   // Token trims them
  }
};

// Logits of one token, its softmax's terms and whether it counts.  cols: E, or
// 0 for a token that does not.
template <typename T, int LPT, int C>
struct Token {
  float z[C][8], x[C][8];         // logits (minus infinity beyond the row), exp(z - m)
  float m, inv;                   // the maximum (0 where all are minus infinity), 1 / sum of x (0 there)
  bool counts;

  __device__ __forceinline__ Token(const Logits<T, LPT, C>& from, int lane, int cols) {
    const float ninf = __uint_as_float(kNegInf);
    float top = ninf;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e0 = (c * LPT + lane) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) z[c][j] = from.raw[c].get(j);
      if (e0 + 8 > cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) z[c][j] = e0 + j < cols ? z[c][j] : ninf;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = __builtin_fmaxf(top, z[c][j]);
    }
    top = lanes_max<LPT>(top);
    counts = top > ninf;
    m = counts ? top : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[c][j] = term(z[c][j]);
        sum += x[c][j];
      }
    sum = lanes_sum<LPT>(sum);
    inv = counts ? 1.0f / sum : 0.0f;
  }
  __device__ __forceinline__ float term(float v) const { return __builtin_amdgcn_exp2f((v - m) * kLog2e); }
};

// in_order(), and 0 for minus infinity and for no number.
__device__ __forceinline__ uint32_t ordered(float v) { return v > __uint_as_float(kNegInf) ? in_order(v) : 0u; }
// The logit of a candidate's key; BF16 keys have the expert in their low half.
__device__ __forceinline__ float logit_of(uint32_t o, float) {
  return __uint_as_float(int32_t(o) < 0 ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ float logit_of(uint32_t o, uint16_t) {
  return __uint_as_float((int32_t(o) < 0 ? o ^ 0x80000000u : ~o) & 0xFFFF0000u);
}

// The larger to the front.
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = a > b ? a : b;
  b = a > b ? b : a;
  a = hi;
}

// Eight in descending order: any, and where the first four and the last four
// make a bitonic sequence.
__device__ __forceinline__ void sort8(uint32_t (&key)[8]) {
  constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                              {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int i = 0; i < 19; ++i) exchange(key[net[i][0]], key[net[i][1]]);   // odd-even merge sort
}
__device__ __forceinline__ void sort8_bitonic(uint32_t (&key)[8]) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) exchange(key[i], key[i + d]);
}

// The eight largest keys of a token in descending order, in every lane of its
// group.  The larger of a[i] and b[7 - i], for two sorted eights a and b, are
// the eight largest of both and bitonic: a level is 8 maxima and 12 exchanges.
template <int LPT, int C>
__device__ __forceinline__ void best_eight(uint32_t (&run)[C][8]) {
  static_assert(C <= 2, "runs of a lane");
  uint32_t(&a)[8] = run[0];
  sort8(a);
  uint32_t o[8];
  const auto join = [&] {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = o[i];
    sort8_bitonic(a);
  };
  if constexpr (C == 2) {
    sort8(run[1]);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = a[i] > run[1][7 - i] ? a[i] : run[1][7 - i];
    join();
  }
  const auto level = [&](auto other) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = other(a[7 - i]);
      o[i] = a[i] > b ? a[i] : b;
    }
    join();
  };
  level([](uint32_t v) { return dpp<0xB1>(v); });  // as in lanes_reduce
  level([](uint32_t v) { return dpp<0x4E>(v); });
  level([](uint32_t v) { return dpp<0x141>(v); });
  if constexpr (LPT >= 16) level([](uint32_t v) { return dpp<0x140>(v); });
  // The swaps give the lower lanes' key first in both halves: the upper ones have the eight in reverse.
  const auto swap_level = [&](auto swap) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const auto v = swap(a[i]);
      lo[i] = v[0];
      hi[i] = v[1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = lo[i] > hi[7 - i] ? lo[i] : hi[7 - i];
    join();
  };
  if constexpr (LPT >= 32) swap_level([](uint32_t v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); });
  if constexpr (LPT >= 64) swap_level([](uint32_t v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); });
}

// A lane's run of eight candidates, experts e0 .. e0 + 7, in descending order.
// BF16 leaves room for the index below the logit: a candidate is one integer, no
// two are equal and a round is one maximum.
template <typename T> struct Run;
template <> struct Run<uint16_t> {
  uint32_t key[8];                // the logit in the high half, 0xFFFF - expert in the low one; 0: none
  __device__ __forceinline__ void sort(const float (&z)[8], int e0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t o = ordered(z[j]);
      key[j] = o ? (o & 0xFFFF0000u) | uint32_t(0xFFFF - (e0 + j)) : 0u;
    }
    sort8(key);
  }
  __device__ __forceinline__ void up(bool taken) {
#pragma unroll
    for (int j = 0; j < 7; ++j) key[j] = taken ? key[j + 1] : key[j];
    key[7] = taken ? 0u : key[7];
  }
};
// FP32: logits, and their places in the run 4 bits each.  Neighbours that are
// equal stay as they are, so that equal logits stay in the order of their index.
template <> struct Run<float> {
  uint32_t key[8];                // 0: none
  uint32_t places;
  __device__ __forceinline__ void sort(const float (&z)[8], int) {
    uint32_t at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      key[j] = ordered(z[j]);
      at[j] = j;
    }
#pragma unroll
    for (int phase = 0; phase < 8; ++phase)
#pragma unroll
      for (int j = phase & 1; j < 7; j += 2) {
        const bool swap = key[j] < key[j + 1];
        exchange(key[j], key[j + 1]);
        const uint32_t x = at[j];
        at[j] = swap ? at[j + 1] : x;
        at[j + 1] = swap ? x : at[j + 1];
      }
    places = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) places |= at[j] << (4 * j);
  }
  __device__ __forceinline__ void up(bool taken) {
#pragma unroll
    for (int j = 0; j < 7; ++j) key[j] = taken ? key[j + 1] : key[j];
    key[7] = taken ? 0u : key[7];
    places = taken ? places >> 4 : places;
  }
};

// One round: the candidate that is chosen, in every lane of the group.
// `key` 0: there is none, `expert` is -1.
struct Choice {
  uint32_t key;
  int expert;
};
template <int LPT, int C>
__device__ __forceinline__ Choice choose(Run<uint16_t> (&run)[C], int) {
  uint32_t best = run[0].key[0];
#pragma unroll
  for (int c = 1; c < C; ++c) best = run[c].key[0] > best ? run[c].key[0] : best;
  best = lanes_max_u32<LPT>(best);
#pragma unroll
  for (int c = 0; c < C; ++c) run[c].up(run[c].key[0] == best);
  return {best, best ? int(0xFFFF - (best & 0xFFFFu)) : -1};
}
template <int LPT, int C>
__device__ __forceinline__ Choice choose(Run<float> (&run)[C], int lane) {
  uint32_t best = run[0].key[0];
#pragma unroll
  for (int c = 1; c < C; ++c) best = run[c].key[0] > best ? run[c].key[0] : best;
  best = lanes_max_u32<LPT>(best);
  uint32_t mine[C], first = 0xFFFFFFFFu;
#pragma unroll
  for (int c = C - 1; c >= 0; --c) {
    mine[c] = uint32_t((c * LPT + lane) * 8) + (run[c].places & 7u);
    first = run[c].key[0] == best ? mine[c] : first;
  }
  first = lanes_min_u32<LPT>(first);
#pragma unroll
  for (int c = 0; c < C; ++c) run[c].up(mine[c] == first);
  return {best, best ? int(first) : -1};
}

// slope of one expert, for n > 0
__device__ __forceinline__ float slope_of(int64_t E, int64_t k, int count, int tokens) {
  return tokens > 0 ? float(E) * float(count) / (float(k) * float(tokens) * float(tokens)) : 0.0f;
}

template <typename T, int LPT, int C, int NT>
__global__ __launch_bounds__(NT) void route_kernel(RouteArgs p) {
  constexpr int G = NT / LPT;                      // tokens at a time
  constexpr int EP = C * LPT * 8;                  // experts with room
  constexpr int ROUNDS = (kMaxChosen + LPT - 1) / LPT;
  __shared__ float sums[NT / 64][EP];
  __shared__ int chosen[EP];
  __shared__ int tokens;
  __shared__ float part[NT / 64];
  const int lane = threadIdx.x & (LPT - 1), group = threadIdx.x / LPT;
  const T* __restrict__ logits = static_cast<const T*>(p.logits);
  const int E = int(p.E), k = int(p.k);
  for (int e = threadIdx.x; e < EP; e += NT) chosen[e] = 0;
  if (threadIdx.x == 0) tokens = 0;
  __syncthreads();
  float acc[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.0f;
  int n = 0;
  // all lanes stay for the exchanges: a group without a token has one that does not count
  for (int64_t t0 = int64_t(blockIdx.x) * G; t0 < p.T; t0 += int64_t(gridDim.x) * G) {
    const int64_t t = t0 + group;
    const bool here = t < p.T;
    Logits<T, LPT, C> z;
    z.load(logits + t * p.ld_z, lane, here ? E : 0);
    const bool valid = here && (!p.valid || p.valid[t] != 0);
    Token<T, LPT, C> tok(z, lane, valid ? E : 0);
    n += tok.counts;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[c][j] = __builtin_fmaf(tok.x[c][j], tok.inv, acc[c][j]);

    float w[ROUNDS], total = 0.0f;                 // lane j of the group has choice r LPT + j
    int ex[ROUNDS];
    bool rounds = k < 4 || k > 8;
    if (!rounds) {
      const uint32_t low = sizeof(T) == 2 ? 0xFFFFu : uint32_t(EP - 1);   // bits of the key that hold the expert
      uint32_t key[C][8];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          key[c][j] = key_of(in_order(tok.z[c][j]), (c * LPT + lane) * 8 + j, low);
      uint32_t(&best)[8] = key[0];
      if constexpr (sizeof(T) == 4) {
        best_eight<LPT, C>(key);
        bool behind = false;
        if (k == 8) {
          const float least = least_of(best[7], low);
          uint32_t n8 = 0;
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) n8 += tok.z[c][j] >= least;
          behind = lanes_reduce<LPT>(n8, [](uint32_t a, uint32_t b) { return a + b; }) > 8;
        }
        rounds = __ballot(tok.counts && (behind || close_among<false>(best, low, k))) != 0;      // uniform over the wave
        if (rounds) {                              // not with logits that have no such bits, as those that were BF16
          uint32_t bits = 0;
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) bits |= __float_as_uint(tok.z[c][j]);
          rounds = __ballot((bits & low) != 0) != 0 && __ballot(tok.counts && (behind || close_among<true>(best, low, k))) != 0;
        }
      } else {
        best_eight<LPT, C>(key);
      }
      uint32_t mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine = lane == j && j < k ? best[j] : mine;
      const bool some = mine >= kLeastKey;
      ex[0] = some ? int(low - (mine & low)) : -1;
      const float z0 = sizeof(T) == 2 ? logit_of(mine, T()) : some ? load1(logits + t * p.ld_z + ex[0]) : 0.0f;
      w[0] = some ? tok.term(z0) * tok.inv : 0.0f;
      total = w[0];
#pragma unroll
      for (int r = 1; r < ROUNDS; ++r) {
        ex[r] = -1;
        w[r] = 0.0f;
      }
    }
    if (rounds) {
      Run<T> run[C];
#pragma unroll
      for (int c = 0; c < C; ++c) run[c].sort(tok.z[c], (c * LPT + lane) * 8);
      total = 0.0f;
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r) {
        uint32_t key = 0;
        ex[r] = -1;
        for (int j = r * LPT; j < k && j < (r + 1) * LPT; ++j) {
          const Choice best = choose<LPT, C>(run, lane);
          if (lane == j - r * LPT) {
            key = best.key;
            ex[r] = best.expert;
          }
        }
        w[r] = key ? tok.term(logit_of(key, T())) * tok.inv : 0.0f;
        total += w[r];
      }
    }
    if (p.renormalize) total = lanes_sum<LPT>(total);
    const float scale = p.renormalize ? (total > 0.0f ? 1.0f / total : 0.0f) : 1.0f;
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int j = r * LPT + lane;
      if (here && j < k) {
        p.weights[t * k + j] = w[r] * scale;
        p.experts[t * k + j] = ex[r];
        if (ex[r] >= 0) atomicAdd(&chosen[ex[r]], 1);      // integers: the order does not matter
      }
    }
  }
  if (lane == 0 && n > 0) atomicAdd(&tokens, n);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = groups_sum<LPT>(acc[c][j]);
      if ((threadIdx.x & 63) < LPT) sums[threadIdx.x >> 6][(c * LPT + lane) * 8 + j] = s;
    }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  float loss = 0.0f;
  for (int e = threadIdx.x; e < E; e += NT) {
    float s = sums[0][e];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) s += sums[w][e];
    if (alone) {
      const float slope = slope_of(p.E, p.k, chosen[e], tokens);
      p.counts[e] = chosen[e];
      p.slope[e] = slope;
      loss = __builtin_fmaf(slope, s, loss);
    } else {
      p.part_p[int64_t(blockIdx.x) * E + e] = s;
      p.part_c[int64_t(blockIdx.x) * E + e] = chosen[e];
    }
  }
  if (alone) {
    loss = row_sum<NT>(loss, part);
    if (threadIdx.x == 0) p.loss[0] = loss;
  } else if (threadIdx.x == 0) {
    p.part_n[blockIdx.x] = tokens;
  }
}

// The tokens that count in all workgroups of the forward kernel, to each of 1024 threads.
__device__ __forceinline__ int tokens_of(const RouteArgs& p, int64_t parts, int* wave_n) {
  int n = 0;
  for (int64_t b = threadIdx.x; b < parts; b += 1024) n += p.part_n[b];
  n = int(lanes_reduce<64>(uint32_t(n), [](uint32_t a, uint32_t b) { return a + b; }));
  if ((threadIdx.x & 63) == 0) wave_n[threadIdx.x >> 6] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) n += wave_n[w];
  return n;
}

// Counts, slopes and the loss by one workgroup: thread t has expert t mod 2^bits
// and takes every (1024 / 2^bits)th of the parts.
__global__ __launch_bounds__(1024) void route_finish_kernel(RouteArgs p, int64_t parts, int bits) {
  __shared__ float sp[1024];
  __shared__ int sc[1024];
  __shared__ int sn[16];
  __shared__ float part[16];
  const int t = threadIdx.x, E = int(p.E), e = t & ((1 << bits) - 1), step = 1024 >> bits;
  float s = 0.0f;
  int c = 0;
  if (e < E) {
#pragma unroll 8
    for (int64_t b = t >> bits; b < parts; b += step) {
      s += p.part_p[b * E + e];
      c += p.part_c[b * E + e];
    }
  }
  sp[t] = s;
  sc[t] = c;
  const int n = tokens_of(p, parts, sn);           // its barrier is also that of sp and sc
  float loss = 0.0f;
  if (t < E) {
    for (int i = t + (1 << bits); i < 1024; i += 1 << bits) {
      s += sp[i];
      c += sc[i];
    }
    const float slope = slope_of(p.E, p.k, c, n);
    p.counts[t] = c;
    p.slope[t] = slope;
    loss = slope * s;
  }
  loss = row_sum<1024>(loss, part);
  if (t == 0) p.loss[0] = loss;
}

// The same for many experts, 64 a workgroup, whose 16 waves take the parts in
// turn; a share of the loss each.
__global__ __launch_bounds__(1024) void route_sums_kernel(RouteArgs p, int64_t parts) {
  __shared__ float sp[16][64];
  __shared__ int sc[16][64];
  __shared__ int sn[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t e = int64_t(blockIdx.x) * 64 + lane;
  float s = 0.0f;
  int c = 0;
  if (e < p.E) {
#pragma unroll 8
    for (int64_t b = wave; b < parts; b += 16) {
      s += p.part_p[b * p.E + e];
      c += p.part_c[b * p.E + e];
    }
  }
  sp[wave][lane] = s;
  sc[wave][lane] = c;
  const int n = tokens_of(p, parts, sn);           // its barrier is also that of sp and sc
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) {
    s += sp[w][lane];
    c += sc[w][lane];
  }
  float slope = 0.0f;
  if (e < p.E) {
    slope = slope_of(p.E, p.k, c, n);
    p.counts[e] = c;
    p.slope[e] = slope;
  }
  const float l = lanes_sum<64>(slope * s);
  if (lane == 0) p.part_l[blockIdx.x] = l;
}

__global__ __launch_bounds__(64) void route_loss_kernel(const float* part, int n, float* loss) {
  const float l = lanes_sum<64>(int(threadIdx.x) < n ? part[threadIdx.x] : 0.0f);
  if (threadIdx.x == 0) *loss = l;
}

template <typename T, int LPT, int C>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBwdArgs p) {
  constexpr int G = 256 / LPT;
  constexpr int ROUNDS = (kMaxChosen + LPT - 1) / LPT;
  const int lane = threadIdx.x & (LPT - 1), group = threadIdx.x / LPT;
  const T* __restrict__ logits = static_cast<const T*>(p.logits);
  T* __restrict__ dlogits = static_cast<T*>(p.dlogits);
  const int E = int(p.E), k = int(p.k);
  const float dloss = p.dloss ? *p.dloss : 0.0f;
  __shared__ __attribute__((aligned(16))) float rows[G][C * LPT * 8];
  float* row = rows[group];                        // of the group's lanes alone, which are in one wave
  float every[C][8];                               // what reaches p of any token
#pragma unroll
  for (int c = 0; c < C; ++c) {
    Row8<float> s;
    load_raw(s, p.slope, (c * LPT + lane) * 8, p.dloss ? E : 0);
    trim(s, (c * LPT + lane) * 8, E);
#pragma unroll
    for (int j = 0; j < 8; ++j) every[c][j] = s.get(j) * dloss;
  }
  for (int64_t t0 = int64_t(blockIdx.x) * G; t0 < p.T; t0 += int64_t(gridDim.x) * G) {
    const int64_t t = t0 + group;
    const bool here = t < p.T;
    Logits<T, LPT, C> z;
    z.load(logits + t * p.ld_z, lane, here ? E : 0);
    int ex[ROUNDS];                                // lane j of the group has choice r LPT + j
    float dc[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int j = r * LPT + lane;
      ex[r] = here && j < k ? p.experts[t * k + j] : -1;
      dc[r] = here && j < k && p.dweights ? p.dweights[t * k + j] : 0.0f;
    }
    const bool counts = __shfl(ex[0], 0, LPT) >= 0;
    Token<T, LPT, C> tok(z, lane, counts ? E : 0);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<v4f*>(row + (c * LPT + lane) * 8 + 4 * q) =
            v4f{every[c][4 * q], every[c][4 * q + 1], every[c][4 * q + 2], every[c][4 * q + 3]};
    wave_order();
    if (p.dweights) {                              // uniform: all lanes exchange
      float pe[ROUNDS], total = 0.0f, dot = 0.0f;
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r) {
        pe[r] = 0.0f;
        if (counts && uint32_t(ex[r]) < uint32_t(E)) {
          if (p.renormalize) pe[r] = tok.term(load1(logits + t * p.ld_z + ex[r])) * tok.inv;
        } else {
          ex[r] = -1;
          dc[r] = 0.0f;
        }
        total += pe[r];
        dot = __builtin_fmaf(dc[r], pe[r], dot);
      }
      if (p.renormalize) {
        total = lanes_sum<LPT>(total);
        dot = lanes_sum<LPT>(dot);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
        const float mean = dot * inv;
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) dc[r] = (dc[r] - mean) * inv;
      }
      // To the experts' places by way of LDS, one after the other, so that an expert that comes more than once has one sum.
      // (Compared with the index of every register in each of the k turns, 8 of 256: BF16 24.5 us, FP32 33.3; so 18.0, 30.0.)
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r)
        for (int j = r * LPT; j < k && j < (r + 1) * LPT; ++j)
          if (lane == j - r * LPT && ex[r] >= 0) atomicAdd(&row[ex[r]], dc[r]);
    }
    wave_order();
    float dp[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const v4f v = *reinterpret_cast<const v4f*>(row + (c * LPT + lane) * 8 + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) dp[c][4 * q + i] = v[i];
      }
    wave_order();
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        tok.x[c][i] *= tok.inv;                    // p
        dot = __builtin_fmaf(tok.x[c][i], dp[c][i], dot);
      }
    dot = lanes_sum<LPT>(dot);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = tok.x[c][i] * (dp[c][i] - dot);
      store_raw(dlogits + t * p.ld_dz, (c * LPT + lane) * 8, here ? E : 0, v);
    }
  }
}

// f(LPT, C) for E experts.  The choice is bound by its instructions: two runs a
// lane share a round's exchanges (65536 tokens, 8 of 256 experts by rounds, FP32:
// 31.6 us with 16 lanes and two runs, 39.1 with 32 and one, 31.3 with 8 and four; 8
// of 512 60 / 81; 8 of 128 17.9 / 20.1).  Lanes: route_lanes().
template <typename F>
hipError_t by_experts(int64_t E, F f) {
  using std::integral_constant;
  if (E <= 64) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
  if (E <= 128) return f(integral_constant<int, 8>(), integral_constant<int, 2>());
  if (E <= 256) return f(integral_constant<int, 16>(), integral_constant<int, 2>());
  if (E <= 512) return f(integral_constant<int, 32>(), integral_constant<int, 2>());
  return f(integral_constant<int, 64>(), integral_constant<int, 2>());
}
// The gradient is bound by memory: as many lanes as there are runs, up to a wave.
template <typename F>
hipError_t by_experts_backward(int64_t E, F f) {
  using std::integral_constant;
  if (E <= 64) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
  if (E <= 128) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
  if (E <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
  if (E <= 512) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
  return f(integral_constant<int, 64>(), integral_constant<int, 2>());
}

template <typename T>
hipError_t launch_route_t(const RouteArgs& p, hipStream_t st) {
  const int64_t parts = route_parts(p.T, p.E);
  const hipError_t e = by_experts(p.E, [&](auto lpt, auto c) {
    const int64_t nt = route_threads(p.T, p.E);
    const dim3 grid{unsigned(parts)};
    if (nt == 256) hipLaunchKernelGGL((route_kernel<T, lpt(), c(), 256>), grid, dim3(256), 0, st, p);
    else if (nt == 512) hipLaunchKernelGGL((route_kernel<T, lpt(), c(), 512>), grid, dim3(512), 0, st, p);
    else hipLaunchKernelGGL((route_kernel<T, lpt(), c(), 1024>), grid, dim3(1024), 0, st, p);
    return hipGetLastError();
  });
  if (e != hipSuccess || parts == 1) return e;
  if (p.E <= 64 || parts * p.E <= kRouteFinish) {
    int bits = 6;
    while ((int64_t(1) << bits) < p.E) ++bits;
    hipLaunchKernelGGL(route_finish_kernel, dim3(1), dim3(1024), 0, st, p, parts, bits);
    return hipGetLastError();
  }
  const unsigned blocks = unsigned((p.E + 63) / 64);
  hipLaunchKernelGGL(route_sums_kernel, dim3(blocks), dim3(1024), 0, st, p, parts);
  const hipError_t e2 = hipGetLastError();
  if (e2 != hipSuccess) return e2;
  hipLaunchKernelGGL(route_loss_kernel, dim3(1), dim3(64), 0, st, p.part_l, int(blocks), p.loss);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_route_backward_t(const RouteBwdArgs& p, hipStream_t st) {
  return by_experts_backward(p.E, [&](auto lpt, auto c) {
    constexpr int64_t G = 256 / decltype(lpt)::value;
    hipLaunchKernelGGL((route_backward_kernel<T, lpt(), c()>), dim3(grid_of((p.T + G - 1) / G, 256)), dim3(256), 0, st, p);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& p, bool bf16, hipStream_t st) {
  return bf16 ? launch_route_t<uint16_t>(p, st) : launch_route_t<float>(p, st);
}
hipError_t launch_moe_route_backward(const RouteBwdArgs& p, bool bf16, hipStream_t st) {
  return bf16 ? launch_route_backward_t<uint16_t>(p, st) : launch_route_backward_t<float>(p, st);
}

}  // namespace fp8q
