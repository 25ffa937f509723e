// Internal launchers behind include/fp8q_front.h, and the sizes of their
// workspaces.  Arguments are validated by abi_front.cpp before any of these is
// called; each enqueues on `st` and returns the launch status without
// synchronising.
#pragma once

#include "../ffn/launch_plan.h"

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fp8q {

// Inputs beyond this many bytes are read past the caches, of which the largest
// holds 256 MB: what is read once would only push out what is read again.
// Smaller ones may still be there from the kernel that wrote them.  Measured (us,
// past the caches / through them): norm of 8192x7168 BF16 with a residual, 235
// MB, inputs just written 78 / 88, from memory 73 / 91; 8192x2048, 67 MB, just
// written 25.0 / 24.6, from memory 27.0 / 32.5, the same inputs again 28.3 / 22.8.
constexpr int64_t kReadOnceBytes = 96 << 20;

struct NormArgs {
  const void* x; int64_t ld_x;
  const void* r; int64_t ld_r;    // or nullptr
  int64_t M, D;
  const void* weight;
  float eps;
  void* h; int64_t ld_h;          // or nullptr
  float* rstd;                    // or nullptr
  void* y; int64_t ld_y;          // or nullptr
  uint8_t* q; int64_t ld_q; float* scales;
  uint8_t* q_t; int64_t ld_qt; float* scales_t;   // or nullptr
  bool once;                      // inputs past the caches
};
hipError_t launch_fp8_rmsnorm(const NormArgs& p, bool x_bf16, bool w_bf16, int mode, hipStream_t st);
hipError_t launch_int8_rmsnorm(const NormArgs& p, bool x_bf16, bool w_bf16, hipStream_t st);

struct NormBwdArgs {
  const void* dy; int64_t ld_dy;
  const void* h; int64_t ld_h;
  int64_t M, D;
  const void* weight;
  const float* rstd;
  const void* dh; int64_t ld_dh;  // or nullptr
  void* dx; int64_t ld_dx;
  float* dw; bool accumulate;
  float* part;                    // [norm_bwd_parts(M, D)][D rounded up to 8]
  bool once;                      // inputs past the caches
};
hipError_t launch_rmsnorm_backward(const NormBwdArgs& p, bool x_bf16, bool w_bf16, hipStream_t st);

// The widest row that a workgroup keeps in registers.
constexpr int64_t kMaxNormD = 32768;

// Rows that a workgroup of the gradient kernel has in hand (a wave each up to
// 1024 channels, 16 lanes up to 256), and workgroups, each of which leaves one
// partial sum of dw per column.  Beyond 256 of them a workgroup takes two rows
// before there are more: the second kernel reads every part (777x2000 FP32, both
// kernels: 12.5 us with 389 workgroups, 12.4 with 256, 14.9 with 777, 14.0 with 128).
inline int64_t norm_bwd_parts(int64_t M, int64_t D) {
  const int64_t rows = D <= 256 ? 16 : D <= 1024 ? 4 : 1, want = M / rows + (M % rows != 0), most = D <= 4096 ? 512 : 256;
  const int64_t half = want / 2 + want % 2, parts = want <= 256 ? want : half > 256 ? half : 256;
  return parts < most ? parts : most;
}
inline int64_t norm_bwd_workspace(int64_t M, int64_t D) { return norm_bwd_parts(M, D) * ((D + 7) / 8 * 8) * 4; }

// ---- routing ---------------------------------------------------------------------

constexpr int64_t kMaxExperts = 1024;
constexpr int kMaxChosen = 32;    // experts of a token

struct RouteArgs {
  const void* logits; int64_t ld_z;
  int64_t T, E, k;
  const uint8_t* valid;           // or nullptr
  bool renormalize;
  float* weights; int32_t* experts; int32_t* counts; float* loss; float* slope;
  float* part_p; int32_t* part_c; int32_t* part_n; float* part_l;   // sums of each workgroup
};
hipError_t launch_moe_route(const RouteArgs& p, bool bf16, hipStream_t st);

struct RouteBwdArgs {
  const void* logits; int64_t ld_z;
  int64_t T, E, k;
  const int32_t* experts; const float* slope;
  const float* dweights; const float* dloss;      // or nullptr
  bool renormalize;
  void* dlogits; int64_t ld_dz;
};
hipError_t launch_moe_route_backward(const RouteBwdArgs& p, bool bf16, hipStream_t st);

// Lanes of a token in the forward kernel.
inline int64_t route_lanes(int64_t E) { return E <= 128 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64; }
// Up to so many tokens (64 of 64 experts, 8 of 1024) one workgroup of 256 threads does it all.
inline int64_t route_few(int64_t E) { return 2 * 256 / route_lanes(E); }
// Threads of a workgroup of the forward kernel, and workgroups.  One alone also
// finishes the sums, in up to two turns of 1024 threads (256 tokens of 64
// experts); more need a second kernel (189 tokens of 9 experts: 9.3 us a call,
// 11.3 in two kernels; with three turns, 384 tokens of 64 experts, 11.4 either way,
// of which the one kernel is 10.8 and the two are 8).  At most 256: each leaves sums
// to be read (65536 tokens of 64 experts, BF16: 12.1 us and 3.8 for the sums, with
// 512 workgroups 13.1 and 4.4).  Their threads: the fewest that take one turn, so
// that all CUs have some (FP32, 8192 tokens: of 64 experts 5.6 us with 256 threads,
// 7.3 with 1024; of 256 experts 8.2 with 512, 12.0).
inline int64_t route_threads(int64_t T, int64_t E) {
  const int64_t all = T * route_lanes(E);
  if (T <= route_few(E)) return 256;
  if (all <= 2 * 1024) return 1024;
  return all <= 256 * 256 ? 256 : all <= 256 * 512 ? 512 : 1024;
}
inline int64_t route_parts(int64_t T, int64_t E) {
  const int64_t all = T * route_lanes(E), nt = route_threads(T, E);
  if (all <= 2 * 1024) return 1;
  return all <= 256 * nt ? (all + nt - 1) / nt : 256;
}
// Sums, one for each part and expert, up to which one workgroup adds them all and the
// loss, beyond 64 experts (one launch / two, us a call and in a graph: 1000 tokens of
// 128 experts, 16128 sums, 14.3 / 17.4 and 9.0 / 9.9; 500 of 512, 32256 sums, 14.1 /
// 17.8 and 12.2 / 11.0; 4096 of 256, 65536 sums, 15.2 / 17.5 and 13.8 / 11.5).
constexpr int64_t kRouteFinish = 32768;
// Sums of p, counts, tokens, and the loss's shares of up to 16 workgroups.
inline int64_t route_workspace(int64_t T, int64_t E) {
  const int64_t parts = route_parts(T, E);
  return parts == 1 ? 0 : parts * E * 8 + (parts + 3) / 4 * 16 + 64;
}

// ---- dispatch --------------------------------------------------------------------

struct DispatchArgs {
  const int32_t* experts;
  int64_t T, k, E;
  const uint8_t* q; int64_t ld_q; const float* scales;
  int64_t D, M_total;
  uint8_t* a; int64_t ld_a; float* a_scales;
  int32_t* group_of_mtile; int32_t* row_of_slot; int32_t* token_of_row;
  int32_t* hist;                  // 17 dispatch_groups(T k) rows of E, or nullptr
};
hipError_t launch_moe_dispatch(const DispatchArgs& p, hipStream_t st);

// Slots that every workgroup counts for itself, in one launch with the rest (us a
// call, in one launch / in two: 16 tokens of 8 experts, 7168 codes, 11.8 / 16.3; 512
// of 8 of 64, 7168 codes 18.0 / 19.8, 2048 codes 13.6 / 16.8; 1024 of 8 of 64, 7168
// codes 40.1 / 29.0, 2048 codes 17.5 / 20.9).
constexpr int64_t kDispatchOneLaunch = 4096;
// Slots whose ranks one workgroup alone finds: a launch less for the host, and one
// CU's work (us a call and in a graph, alone / in two kernels: 4352 slots of 8 of 64
// experts, 128 codes, 16.0 / 15.9 and 15.2 / 14.0, 2048 codes 18.2 / 18.2 and 18.0 /
// 16.7; of 2 of 8, 128 codes, 14.5 / 16.4 and 13.9 / 13.7; 8192 slots of 8 of 64, 128
// codes, 17.9 / 15.8 and 17.3 / 14.0, 7168 codes 30.3 / 27.5 and 30.6 / 27.4; of 8 of
// 256, 2048 codes, 28.4 / 25.2 and 28.4 / 25.4).  It is ahead up to some 5000 slots
// where the host is what a call waits for, and behind elsewhere.
constexpr int64_t kDispatchAlone = 8192;

// Slots of one wave, whole steps of 64, for up to 128 workgroups of 16 waves.
inline int64_t dispatch_chunk(int64_t slots) {
  const int64_t steps = (slots + 64 * 16 * 128 - 1) / (64 * 16 * 128);
  return 64 * (steps > 2 ? steps : 2);
}
inline int64_t dispatch_groups(int64_t slots) {
  return slots <= kDispatchAlone ? 0 : (slots - 1) / (16 * dispatch_chunk(slots)) + 1;
}
inline int64_t dispatch_workspace(int64_t slots, int64_t E) { return dispatch_groups(slots) * 17 * E * 4; }

// Whole 128-row tiles that the slots take at most: each of n experts wastes up to 127 rows.
inline int64_t dispatch_max_rows(int64_t slots, int64_t E) {
  return (slots + 127 * (slots < E ? slots : E)) / 128 * 128;
}

}  // namespace fp8q
