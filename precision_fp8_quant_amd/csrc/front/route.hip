// The k experts of each token, their weights, the tokens of each expert and the
// loss that balances them; and the gradient with respect to the logits.
//
//   p = softmax(z);  loss = sum_e slope_e sum_t p_te,  slope_e = E c_e / (k n^2)
//   dz = p (dp - sum p dp),  dp_e = dloss slope_e + [e chosen] dc
// LPT lanes share a token and hold its logits in registers, C runs of 8 each
// (expert (c LPT + lane) 8 + j): one read of the logits serves the softmax and
// the choice.  The choice is k rounds of a maximum over the lanes and of the
// lowest index that has it, on the logits themselves, so that equal logits are
// equal.
//
// A lane has the same 8 C experts in all of its workgroup's tokens and sums
// their p in registers, a wave its groups', a workgroup its waves'; workgroups
// leave one row of sums and counts each, which a second kernel adds in a fixed
// order.  With one workgroup it is all one launch.
#include "front_launch.h"
#include "lanes.h"
#include "row_io.h"

#include <type_traits>

namespace fp8q {
namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr uint32_t kNegInf = 0xFF800000u;

// Logits of one token, its softmax's terms and whether it counts.  cols: E, or
// 0 for a token whose logits are not read.
template <typename T, int LPT, int C>
struct Token {
  float z[C][8], x[C][8];         // logits (minus infinity beyond the row), exp(z - m)
  float m, inv;                   // the maximum (0 where all are minus infinity), 1 / sum of x (0 there)
  bool counts;

  __device__ __forceinline__ void load(const T* row, int lane, int cols) {
    const float ninf = __uint_as_float(kNegInf);
    float top = ninf;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e0 = (c * LPT + lane) * 8;
      Row8<T> raw;
      load_raw(raw, row, e0, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[c][j] = e0 + j < cols ? raw.get(j) : ninf;
        top = __builtin_fmaxf(top, z[c][j]);
      }
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

// slope of one expert, for n > 0
__device__ __forceinline__ float slope_of(int64_t E, int64_t k, int count, int tokens) {
  return tokens > 0 ? float(E) * float(count) / (float(k) * float(tokens) * float(tokens)) : 0.0f;
}

// v summed over the lanes that have the same place in their group of LPT.
template <int LPT>
__device__ __forceinline__ float groups_sum(float v) {
  if constexpr (LPT <= 8) v += __uint_as_float(dpp<0x128>(__float_as_uint(v)));        // row_ror by 8: the other half row
  if constexpr (LPT <= 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(uint32_t(a[0])) + __uint_as_float(uint32_t(a[1]));
  }
  if constexpr (LPT <= 32) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(uint32_t(a[0])) + __uint_as_float(uint32_t(a[1]));
  }
  return v;
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
    const bool read = here && (!p.valid || p.valid[t] != 0);
    Token<T, LPT, C> tok;
    tok.load(logits + t * p.ld_z, lane, read ? E : 0);
    n += tok.counts;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[c][j] = __builtin_fmaf(tok.x[c][j], tok.inv, acc[c][j]);

    float w[ROUNDS], total = 0.0f;
    int ex[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      w[r] = 0.0f;
      ex[r] = -1;
      for (int j = r * LPT; j < k && j < (r + 1) * LPT; ++j) {
        float best = __uint_as_float(kNegInf);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) best = __builtin_fmaxf(best, tok.z[c][i]);
        best = lanes_max<LPT>(best);
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int c = C - 1; c >= 0; --c)
#pragma unroll
          for (int i = 7; i >= 0; --i)
            at = tok.z[c][i] == best ? uint32_t((c * LPT + lane) * 8 + i) : at;
        at = lanes_min_u32<LPT>(at);
        const bool found = best > __uint_as_float(kNegInf);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            tok.z[c][i] = at == uint32_t((c * LPT + lane) * 8 + i) ? __uint_as_float(kNegInf) : tok.z[c][i];
        const float wj = found ? tok.term(best) * tok.inv : 0.0f;
        total += wj;
        if (lane == j - r * LPT) {
          w[r] = wj;
          ex[r] = found ? int(at) : -1;
        }
      }
    }
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

// Counts, slopes and the loss's share of 64 experts a workgroup: 16 waves take
// the parts in turn.  `loss`: the loss itself where this is the only workgroup,
// one word for each otherwise.
__global__ __launch_bounds__(1024) void route_sums_kernel(RouteArgs p, int64_t parts, float* loss) {
  __shared__ float sp[16][64];
  __shared__ int sc[16][64];
  __shared__ int sn[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t e = int64_t(blockIdx.x) * 64 + lane;
  int n = 0;
  for (int64_t b = threadIdx.x; b < parts; b += 1024) n += p.part_n[b];
  n = int(lanes_reduce<64>(uint32_t(n), [](uint32_t a, uint32_t b) { return a + b; }));
  if (lane == 0) sn[wave] = n;
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
  __syncthreads();
  if (wave != 0) return;
  n = sn[0];
#pragma unroll
  for (int w = 1; w < 16; ++w) {
    n += sn[w];
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
  if (lane == 0) loss[blockIdx.x] = l;
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
  float every[C][8];                               // what reaches p of any token
#pragma unroll
  for (int c = 0; c < C; ++c) {
    Row8<float> s;
    load_raw(s, p.slope, (c * LPT + lane) * 8, p.dloss ? E : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) every[c][j] = s.get(j) * dloss;
  }
  for (int64_t t0 = int64_t(blockIdx.x) * G; t0 < p.T; t0 += int64_t(gridDim.x) * G) {
    const int64_t t = t0 + group;
    const bool here = t < p.T;
    const bool counts = here && p.experts[t * k] >= 0;
    Token<T, LPT, C> tok;
    tok.load(logits + t * p.ld_z, lane, counts ? E : 0);
    float dp[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) dp[c][j] = every[c][j];
    if (p.dweights) {                              // uniform: all lanes exchange
      int ex[ROUNDS];
      float dc[ROUNDS], pe[ROUNDS], total = 0.0f, dot = 0.0f;
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r) {
        const int j = r * LPT + lane;
        ex[r] = -1;
        dc[r] = pe[r] = 0.0f;
        if (counts && j < k) {
          const int e = p.experts[t * k + j];
          if (e >= 0 && e < E) {
            ex[r] = e;
            dc[r] = p.dweights[t * k + j];
            if (p.renormalize) pe[r] = tok.term(load1(logits + t * p.ld_z + e)) * tok.inv;
          }
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
#pragma unroll
      for (int r = 0; r < ROUNDS; ++r)
        for (int j = r * LPT; j < k && j < (r + 1) * LPT; ++j) {
          const int e = __shfl(ex[r], j - r * LPT, LPT);
          const float d = __shfl(dc[r], j - r * LPT, LPT);
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) dp[c][i] += e == (c * LPT + lane) * 8 + i ? d : 0.0f;
        }
    }
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

// f(LPT, C) for E experts
template <typename F>
hipError_t by_experts(int64_t E, F f) {
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
    if (parts == 1) hipLaunchKernelGGL((route_kernel<T, lpt(), c(), 256>), dim3(1), dim3(256), 0, st, p);
    else hipLaunchKernelGGL((route_kernel<T, lpt(), c(), 1024>), dim3(unsigned(parts)), dim3(1024), 0, st, p);
    return hipGetLastError();
  });
  if (e != hipSuccess || parts == 1) return e;
  const unsigned blocks = unsigned((p.E + 63) / 64);
  hipLaunchKernelGGL(route_sums_kernel, dim3(blocks), dim3(1024), 0, st, p, parts, blocks == 1 ? p.loss : p.part_l);
  const hipError_t e2 = hipGetLastError();
  if (e2 != hipSuccess || blocks == 1) return e2;
  hipLaunchKernelGGL(route_loss_kernel, dim3(1), dim3(64), 0, st, p.part_l, int(blocks), p.loss);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_route_backward_t(const RouteBwdArgs& p, hipStream_t st) {
  return by_experts(p.E, [&](auto lpt, auto c) {
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
