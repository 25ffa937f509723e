// Rows of codes in the order of their experts, each expert's rows padded to
// whole 128-row tiles.
//
//   s_e = 128 sum_{i<e} ceil(c_i / 128),  row(t, j) = s_e + slots of e before (t, j)
// The order within an expert is the order of the slots (t k + j), so the result
// does not depend on timing.  A wave takes a chunk of slots 64 at a time: lanes
// of equal experts find each other by one ballot per bit of the expert, a
// lane's place is the expert's running count plus its equals in lower lanes.
//   up to 4096 slots   no plan of its own: every workgroup of the one kernel finds
//                      the experts' tiles and its tile's tokens for itself
//   up to 8192         one workgroup: counts of its 16 waves' chunks, their
//                      prefix sums and the tile map, the rows
//   beyond             two kernels of up to 128 workgroups of 16 chunks: the counts
//                      of chunks and workgroups; then the rows, every workgroup
//                      summing the others' counts for itself
// Then (beyond 4096 slots) one kernel moves codes and scales: a token's row is
// read once and written to its k places; scales, which lie transposed, are
// written in runs of a tile's 128 rows, with the padding rows of the tile.
// Bound by memory: 65536 rows of 7168 codes move in 117 us, 5.0 TB/s (a large copy:
// 5.1), after 11 us of plan; 128 slots of 64 experts take 12 us, of which 38 MB are
// zeros of padding.
#include "front_launch.h"
#include "lanes.h"
#include "row_io.h"

namespace fp8q {
namespace {

constexpr uint32_t kZeroScaleBits = 0x00800000u;   // 2^-126: the scale of a row of zeros

constexpr int kSteps = 4;     // steps of 64 slots whose experts a wave loads together

// The experts of slots [s, s + 64 kSteps) up to `end`, a lane's at s + 64 i + lane; -1 for no expert.
__device__ __forceinline__ void load_experts(const DispatchArgs& p, int64_t s, int64_t end, int (&e)[kSteps]) {
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t slot = s + 64 * i + (threadIdx.x & 63);
    e[i] = slot < end ? p.experts[slot] : -1;
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) e[i] = uint32_t(e[i]) < uint32_t(p.E) ? e[i] : -1;
}

// Adds the experts of slots [begin, end) to count[], by one wave.
__device__ __forceinline__ void count_chunk(const DispatchArgs& p, int64_t begin, int64_t end, int* count) {
  for (int64_t s = begin; s < end; s += 64 * kSteps) {
    int e[kSteps];
    load_experts(p, s, end, e);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (e[i] >= 0) atomicAdd(&count[e[i]], 1);   // integers: the order does not matter
  }
}

// The rows of slots [begin, end), by one wave, whose first experts are in e;
// next[x] is expert x's next row, in LDS that no other wave writes.
__device__ __forceinline__ void place_chunk(const DispatchArgs& p, int64_t begin, int64_t end, int bits, int* next,
                                            int (&e)[kSteps]) {
  const int lane = threadIdx.x & 63;
  const uint64_t below_mask = (uint64_t(1) << lane) - 1;
  for (int64_t s = begin; s < end; s += 64 * kSteps) {     // uniform over the wave
    if (s > begin) load_experts(p, s, end, e);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t slot = s + 64 * i + lane;
      if (s + 64 * i >= end) break;                // uniform over the wave
      uint64_t same = __ballot(e[i] >= 0);
      for (int b = 0; b < bits; ++b) {
        const bool set = (e[i] >> b) & 1;
        const uint64_t one = __ballot(set);
        same &= set ? one : ~one;
      }
      const uint64_t below = same & below_mask;
      int row = -1;
      if (e[i] >= 0) row = next[e[i]] + __popcll(below);
      wave_order();                                // the wave's reads come before its writes
      if (e[i] >= 0 && below == 0) next[e[i]] = row + __popcll(same);
      wave_order();
      if (slot < end) p.row_of_slot[slot] = row;
      if (e[i] >= 0) p.token_of_row[row] = int32_t(slot / p.k);
    }
  }
}

// Exclusive sums over the workgroup's 1024 threads; *total is the sum.
__device__ __forceinline__ int block_exclusive(int v, int* wave_sum, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  if (lane == 63) wave_sum[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    before += w < wave ? wave_sum[w] : 0;
    all += wave_sum[w];
  }
  *total = all;
  return before + s - v;
}

// The tile map and the rows that hold no token, by 1024 threads: thread e < E
// has expert e's count and first tile.
__device__ __forceinline__ void write_maps(const DispatchArgs& p, int count, int first, int tiles_used, int (*place)[2]) {
  const int t = threadIdx.x, tiles = int(p.M_total >> 7), E = int(p.E);
  if (t < E) {
    place[t][0] = first * 128 + count;             // padding rows: [0] to [1]
    place[t][1] = (first + ((count + 127) >> 7)) * 128;
  }
  for (int i = tiles_used + t; i < tiles; i += 1024) p.group_of_mtile[i] = -1;
  for (int64_t i = int64_t(tiles_used) * 128 + t; i < p.M_total; i += 1024) p.token_of_row[i] = -1;
  __syncthreads();
  for (int i = t; i < tiles_used; i += 1024) {     // the first expert that ends behind the tile's first row
    int lo = 0, hi = E - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (place[mid][1] > i * 128) hi = mid;
      else lo = mid + 1;
    }
    p.group_of_mtile[i] = lo;
  }
  for (int i = t; i < E * 128; i += 1024) {
    const int row = place[i >> 7][0] + (i & 127);
    if (row < place[i >> 7][1]) p.token_of_row[row] = -1;
  }
}

__global__ __launch_bounds__(1024) void plan_kernel(DispatchArgs p, int chunk, int bits) {
  __shared__ int next[16][kMaxExperts];
  __shared__ int place[kMaxExperts][2];
  __shared__ int wave_sum[16];
  const int t = threadIdx.x, wave = t >> 6, E = int(p.E);
  const int64_t slots = p.T * p.k, begin = int64_t(wave) * chunk;
  const int64_t end = begin + chunk < slots ? begin + chunk : slots;
  for (int e = t & 63; e < E; e += 64) next[wave][e] = 0;
  __syncthreads();
  int first_experts[kSteps];
  load_experts(p, begin, end, first_experts);
  count_chunk(p, begin, end, next[wave]);
  __syncthreads();
  int count = 0;
  if (t < E) {
#pragma unroll
    for (int w = 0; w < 16; ++w) count += next[w][t];
  }
  int used;
  const int first = block_exclusive((count + 127) >> 7, wave_sum, &used);
  if (t < E) {
    int row = first * 128;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      const int c = next[w][t];
      next[w][t] = row;
      row += c;
    }
  }
  write_maps(p, count, first, used, place);        // its barrier is also that of next[]
  place_chunk(p, begin, end, bits, next[wave], first_experts);
}

// hist: the counts of each chunk, [chunks][E], then those of each workgroup.
__global__ __launch_bounds__(1024) void plan_count_kernel(DispatchArgs p, int64_t chunk) {
  __shared__ int count[16][kMaxExperts];
  const int t = threadIdx.x, wave = t >> 6, E = int(p.E);
  const int64_t c = int64_t(blockIdx.x) * 16 + wave, chunks = int64_t(gridDim.x) * 16;
  for (int e = t & 63; e < E; e += 64) count[wave][e] = 0;
  __syncthreads();
  const int64_t slots = p.T * p.k, end = (c + 1) * chunk < slots ? (c + 1) * chunk : slots;
  count_chunk(p, c * chunk, end, count[wave]);
  __syncthreads();
  for (int e = t & 63; e < E; e += 64) p.hist[c * E + e] = count[wave][e];
  if (t < E) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) n += count[w][t];
    p.hist[(chunks + blockIdx.x) * E + t] = n;
  }
}

// Up to 16 threads (1024 over E rounded up to a power of two) sum an expert's
// counts over consecutive pieces of the workgroups: all of them for the first
// rows of the experts, those before this one for its own.  One workgroup more
// than there are of chunks writes the maps.
__global__ __launch_bounds__(1024) void plan_place_kernel(DispatchArgs p, int64_t chunk, int bits) {
  __shared__ int next[16][kMaxExperts];
  __shared__ int place[kMaxExperts][2];
  __shared__ int wave_sum[16];
  int* sums = next[0];                             // [2][1024], before next[] is filled
  const int t = threadIdx.x, wave = t >> 6, E = int(p.E), ep = 1 << bits, share = bits < 6 ? 16 : 1024 >> bits;
  const int blocks = int(gridDim.x) - 1, mine = blockIdx.x;
  const int64_t c = int64_t(mine) * 16 + wave, slots = p.T * p.k, begin = c * chunk;
  const int64_t end = begin + chunk < slots ? begin + chunk : slots;
  const int* group_counts = p.hist + int64_t(blocks) * 16 * E;
  int experts[kSteps];
  load_experts(p, begin, end, experts);
  const int e = t & (ep - 1), piece = t >> bits, len = (blocks + share - 1) / share;
  const int c0 = piece * len, c1 = c0 + len < blocks ? c0 + len : blocks;
  int all = 0, before = 0;
  if (e < E && piece < share) {
#pragma unroll 4
    for (int i = c0; i < c1; ++i) {
      const int n = group_counts[int64_t(i) * E + e];
      all += n;
      before += i < mine ? n : 0;
    }
  }
  int own[16];
  if (t < E && mine < blocks) {
#pragma unroll
    for (int w = 0; w < 16; ++w) own[w] = p.hist[(int64_t(mine) * 16 + w) * E + t];
  }
  sums[t] = all;
  sums[1024 + t] = before;
  __syncthreads();
  all = before = 0;
  if (t < E)
    for (int s = 0; s < share; ++s) {
      all += sums[s * ep + t];
      before += sums[1024 + s * ep + t];
    }
  int used;
  const int first = block_exclusive((all + 127) >> 7, wave_sum, &used);   // its barrier: sums[] has been read
  if (mine == blocks) {                            // uniform over the workgroup
    write_maps(p, all, first, used, place);
    return;
  }
  if (t < E) {
    int row = first * 128 + before;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      next[w][t] = row;
      row += own[w];
    }
  }
  __syncthreads();
  place_chunk(p, begin, end, bits, next[wave], experts);
}

// Work units: first every tile in pieces of 16 groups (2048 codes of a row),
// then every token in pieces of 1024 codes, one wave each (65536 rows of 7168 codes,
// alone, us: 120; a wave for a whole row 127, a workgroup for one 123, a wave for each
// row of a, which reads a token's row k times, 142; codes read through the caches 128).
__global__ __launch_bounds__(256) void move_kernel(DispatchArgs p, int64_t tile_units, int64_t blocks) {
  __shared__ int token[128];
  const int t = threadIdx.x;
  const int64_t groups = p.D >> 7;
  for (int64_t u = blockIdx.x; u < blocks; u += gridDim.x) {     // block-uniform: barriers stay matched
    if (u < tile_units) {
      const int64_t pieces = (groups + 15) >> 4, tile = u / pieces, g0 = u % pieces * 16;
      if (p.group_of_mtile[tile] < 0) continue;
      const int64_t g1 = g0 + 16 < groups ? g0 + 16 : groups;
      const int mine = p.token_of_row[tile * 128 + (t & 127)];
      __syncthreads();                             // token[] may still be read for the last tile
      if (t < 128) token[t] = mine;
      __syncthreads();
      for (int64_t g = g0 + (t >> 7); g < g1; g += 2)
        p.a_scales[g * p.M_total + tile * 128 + (t & 127)] =
            mine >= 0 ? p.scales[g * p.T + mine] : __uint_as_float(kZeroScaleBits);
      const int64_t col = g0 * 128 + (t & 127) * 16;
      if (col < p.D)
        for (int r = t >> 7; r < 128; r += 2)
          if (token[r] < 0) *reinterpret_cast<u32x4*>(p.a + (tile * 128 + r) * p.ld_a + col) = u32x4{0u, 0u, 0u, 0u};
    } else {
      const int64_t pieces = (p.D + 1023) >> 10, w = (u - tile_units) * 4 + (t >> 6);
      const int64_t tok = w / pieces, col = (w % pieces) * 1024 + (t & 63) * 16;
      if (tok >= p.T || col >= p.D) continue;
      const u32x4 v = load_vec<true, u32x4>(p.q + tok * p.ld_q + col);
      for (int j = 0; j < int(p.k); ++j) {
        const int row = p.row_of_slot[tok * p.k + j];
        if (row >= 0) *reinterpret_cast<u32x4*>(p.a + row * p.ld_a + col) = v;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Few slots, as in a decode batch, whose bytes are mostly padding: one launch,
// work units of a tile's rows by 1024 codes.  Each workgroup counts all slots,
// finds the expert of its tile and lists the tile's slots in their order; the
// first piece of a tile also writes its part of the maps.
// ---------------------------------------------------------------------------
template <int STEPS>                                // slots of a thread; a wave's are consecutive
__global__ __launch_bounds__(256) void dispatch_few_kernel(DispatchArgs p, int64_t pieces, int64_t units) {
  constexpr int PER = int(kMaxExperts) / 256;      // experts of a thread
  __shared__ int count[kMaxExperts];
  __shared__ int token[128], slot_of[128];
  __shared__ int wave_sum[4];
  __shared__ int tile_expert, tile_skip;           // the tile's expert (-1: not in use), its slots in earlier tiles
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, E = int(p.E), slots = int(p.T * p.k), k = int(p.k);
  const int slot0 = wave * (STEPS * 64) + lane;
  int e[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int s = slot0 + 64 * i;
    e[i] = s < slots ? p.experts[s] : -1;
  }
  for (int x = t; x < int(kMaxExperts); x += 256) count[x] = 0;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) e[i] = uint32_t(e[i]) < uint32_t(E) ? e[i] : -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (e[i] >= 0) atomicAdd(&count[e[i]], 1);     // integers: the order does not matter
  __syncthreads();
  // tiles before each of the thread's experts
  int n[PER], mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    n[i] = (count[t * PER + i] + 127) >> 7;
    mine += n[i];
  }
  int before = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(before, d, 64);
    if (lane >= d) before += o;
  }
  if (lane == 63) wave_sum[wave] = before;
  __syncthreads();
  before -= mine;
  for (int w = 0; w < wave; ++w) before += wave_sum[w];

  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {      // block-uniform: barriers stay matched
    const int tile = int(u / pieces), piece = int(u % pieces);
    if (u == 0) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        if (slot0 + 64 * i < slots && e[i] < 0) p.row_of_slot[slot0 + 64 * i] = -1;
    }
    if (t == 0) tile_expert = -1;
    if (t < 128) token[t] = -1;
    __syncthreads();
    int first = before;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (tile >= first && tile < first + n[i]) {  // one thread's, for one expert
        tile_expert = t * PER + i;
        tile_skip = (tile - first) * 128;
      }
      first += n[i];
    }
    __syncthreads();
    const int expert = tile_expert, skip = tile_skip;
    // the expert's slots in the waves before this one, then one by one
    int at = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) at += __popcll(__ballot(expert >= 0 && e[i] == expert));
    if (lane == 0) wave_sum[wave] = at;
    __syncthreads();
    at = -skip;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const bool hit = expert >= 0 && e[i] == expert;
      const uint64_t all = __ballot(hit);
      const int r = at + __popcll(all & ((uint64_t(1) << lane) - 1));
      if (hit && r >= 0 && r < 128) {
        token[r] = (slot0 + 64 * i) / k;
        slot_of[r] = slot0 + 64 * i;
      }
      at += __popcll(all);
    }
    __syncthreads();
    if (piece == 0) {
      if (t == 0) p.group_of_mtile[tile] = expert;
      if (t < 128) {
        p.token_of_row[tile * 128 + t] = token[t];
        if (token[t] >= 0) p.row_of_slot[slot_of[t]] = tile * 128 + t;
      }
    }
    if (expert >= 0) {
      const int64_t groups = p.D >> 7, g0 = int64_t(piece) * 8, g1 = g0 + 8 < groups ? g0 + 8 : groups;
      const int row = t & 127, tok = token[row];
      for (int64_t g = g0 + (t >> 7); g < g1; g += 2)
        p.a_scales[g * p.M_total + tile * 128 + row] = tok >= 0 ? p.scales[g * p.T + tok] : __uint_as_float(kZeroScaleBits);
      const int64_t col = int64_t(piece) * 1024 + lane * 16;
      if (col < p.D) {
#pragma unroll 8
        for (int r = wave; r < 128; r += 4) {
          u32x4 v = {0u, 0u, 0u, 0u};
          if (token[r] >= 0) v = *reinterpret_cast<const u32x4*>(p.q + token[r] * p.ld_q + col);
          *reinterpret_cast<u32x4*>(p.a + (int64_t(tile) * 128 + r) * p.ld_a + col) = v;
        }
      }
    }
    __syncthreads();                               // token[] and wave_sum[] are written again for the next unit
  }
}

int bits_of(int64_t E) {                           // bits that tell E experts apart
  int b = 0;
  while ((int64_t(1) << b) < E) ++b;
  return b;
}

}  // namespace

hipError_t launch_moe_dispatch(const DispatchArgs& p, hipStream_t st) {
  const int64_t slots = p.T * p.k;
  if (slots <= kDispatchOneLaunch) {
    const int64_t pieces = p.D > 1024 ? (p.D + 1023) / 1024 : 1, units = p.M_total / 128 * pieces;
    const dim3 grid(grid_of(units, 256));
    if (slots <= 1024) hipLaunchKernelGGL(dispatch_few_kernel<4>, grid, dim3(256), 0, st, p, pieces, units);
    else hipLaunchKernelGGL(dispatch_few_kernel<kDispatchOneLaunch / 256>, grid, dim3(256), 0, st, p, pieces, units);
    return hipGetLastError();
  }
  const unsigned groups = unsigned(dispatch_groups(slots));
  const int bits = bits_of(p.E);
  if (groups == 0) {
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(1024), 0, st, p, int((slots + 1023) / 1024 * 64), bits);
  } else {
    const int64_t chunk = dispatch_chunk(slots);
    hipLaunchKernelGGL(plan_count_kernel, dim3(groups), dim3(1024), 0, st, p, chunk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(plan_place_kernel, dim3(groups + 1), dim3(1024), 0, st, p, chunk, bits);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.T == 0 || p.D == 0) return e;
  const int64_t tile_units = (p.M_total / 128) * ((p.D / 128 + 15) / 16);
  const int64_t blocks = tile_units + (p.T * ((p.D + 1023) / 1024) + 3) / 4;
  hipLaunchKernelGGL(move_kernel, dim3(grid_of(blocks, 256)), dim3(256), 0, st, p, tile_units, blocks);
  return hipGetLastError();
}

}  // namespace fp8q
