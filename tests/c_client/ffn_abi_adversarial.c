/*
 * Argument validation of include/fp8q_ffn.h from plain C against adversarial
 * sizes, leading dimensions and addresses.  Linked with abi_ffn.cpp and host
 * stand-ins for the launchers (no GPU): every call must return its documented
 * status, and a request that passes validation must reach exactly one launcher.
 */
#include <stdint.h>
#include <stdio.h>

#include "fp8q_ffn.h"

extern int fp8q_ffn_stub_launches;

static int failures = 0;

static void expect(int line, int got, int want, int launches) {
  static int seen = 0;
  if (got != want || fp8q_ffn_stub_launches - seen != launches) {
    fprintf(stderr, "line %d: status %d, expected %d; %d launches\n", line, got, want, fp8q_ffn_stub_launches - seen);
    ++failures;
  }
  seen = fp8q_ffn_stub_launches;
}

#define EXPECT(call, want) expect(__LINE__, (call), (want), 0)
#define LAUNCHES(call) expect(__LINE__, (call), FP8Q_OK, 1)

int main(void) {
  /* plausible, aligned, disjoint fake device addresses (never dereferenced) */
  uint8_t* A = (uint8_t*)(uintptr_t)0x10000000000ull;
  float* B = (float*)(uintptr_t)0x20000000000ull;
  uint8_t* C = (uint8_t*)(uintptr_t)0x30000000000ull;
  float* D = (float*)(uintptr_t)0x40000000000ull;
  uint8_t* E = (uint8_t*)(uintptr_t)0x50000000000ull;
  float* F = (float*)(uintptr_t)0x60000000000ull;
  void* G = (void*)(uintptr_t)0x70000000000ull;
  /* 16-byte aligned, 64 bytes below the top of the address space */
  void* TOP = (void*)(uintptr_t)(UINTPTR_MAX - 63u);
  const int64_t MAX = INT64_MAX, BIG = INT64_MAX / 256 * 128, LD = INT64_MAX / 8 / 16 * 16;
  const int8_t* a8 = (const int8_t*)A;
  const int8_t* c8 = (const int8_t*)C;

  LAUNCHES(fp8_gemm_gated(0, 1, 128, 128, A, 128, B, C, 128, D, E, FP8Q_BF16, 128, G, 256, NULL));
  LAUNCHES(fp8_gemm_gated(1, 3, 128, 0, NULL, 0, NULL, NULL, 0, NULL, E, FP8Q_F32, 128, NULL, 0, NULL));
  LAUNCHES(fp8_gated_backward(0, 1, 128, A, 128, C, 256, FP8Q_F32, 1, E, 256, B, (uint8_t*)G, 128, F, NULL, 0, NULL));
  LAUNCHES(int8_quant_rows(A, FP8Q_F32, 3, 5, 8, (int8_t*)C, 16, B, NULL));
  LAUNCHES(int8_quant_rows(NULL, FP8Q_F32, 3, 0, 0, NULL, 0, B, NULL));
  LAUNCHES(int8_gemm(1, 1, 1, a8, 16, B, c8, 16, D, NULL, E, FP8Q_F32, 4, NULL));
  LAUNCHES(int8_gemm_gated(1, 2, 3, 131056, a8, 131056, B, c8, 131056, D, E, FP8Q_BF16, 8, NULL));

  /* sizes whose doubles, extents or counts overflow */
  EXPECT(fp8_gemm_gated(0, 1, BIG, 128, A, 128, B, C, 128, D, E, FP8Q_BF16, BIG, NULL, 0, NULL), FP8Q_ERR_UNSUPPORTED);
  EXPECT(fp8_gemm_gated(0, 1, MAX / 128 * 128, 128, A, 128, B, C, 128, D, E, FP8Q_BF16, MAX, NULL, 0, NULL),
         FP8Q_ERR_SHAPE);
  EXPECT(fp8_gemm_gated(0, MAX, 128, 128, A, 128, B, C, 128, D, E, FP8Q_BF16, 128, NULL, 0, NULL),
         FP8Q_ERR_UNSUPPORTED);
  EXPECT(fp8_gemm_gated(0, 1 << 20, 128, 128, A, 128, B, C, 128, D, E, FP8Q_F32, LD, NULL, 0, NULL), FP8Q_ERR_SHAPE);
  EXPECT(fp8_gemm_gated(0, 40, 128, 128, A, 128, B, C, 128, D, E, FP8Q_BF16, 128, G, LD, NULL), FP8Q_ERR_SHAPE);
  EXPECT(fp8_gemm_gated(0, 4, 128, 128, A, 128, B, C, 128, D, TOP, FP8Q_BF16, 128, NULL, 0, NULL), FP8Q_ERR_SHAPE);
  EXPECT(fp8_gemm_gated(0, 4, 128, 128, (uint8_t*)TOP, 128, B, C, 128, D, E, FP8Q_BF16, 128, NULL, 0, NULL),
         FP8Q_ERR_SHAPE);
  EXPECT(fp8_gated_backward(0, MAX, 128, A, 128, C, 256, FP8Q_F32, 1, E, 256, B, (uint8_t*)G, MAX, F, NULL, 0, NULL),
         FP8Q_ERR_SHAPE);
  EXPECT(fp8_gated_backward(0, 8, MAX / 2 + 1, A, MAX, C, MAX, FP8Q_F32, 1, E, MAX, B, (uint8_t*)G, 128, F, NULL, 0,
                            NULL), FP8Q_ERR_SHAPE);
  EXPECT(fp8_gated_backward(0, 300, 128, A, LD, C, 256, FP8Q_F32, 1, E, 256, B, (uint8_t*)G, 384, F, NULL, 0, NULL),
         FP8Q_ERR_SHAPE);
  EXPECT(fp8_gated_backward(0, 300, 128, A, 128, C, 256, FP8Q_F32, 1, E, 256, B, (uint8_t*)G, 384, F, TOP, 256, NULL),
         FP8Q_ERR_SHAPE);
  EXPECT(int8_quant_rows(A, FP8Q_F32, MAX, MAX, MAX, (int8_t*)C, MAX, B, NULL), FP8Q_ERR_ALIGN);
  EXPECT(int8_quant_rows(A, FP8Q_F32, MAX, 16, 16, (int8_t*)C, 16, B, NULL), FP8Q_ERR_SHAPE);
  EXPECT(int8_quant_rows(A, FP8Q_BF16, 32, 16, 16, (int8_t*)C, 16, (float*)TOP, NULL), FP8Q_ERR_SHAPE);
  EXPECT(int8_gemm(MAX, MAX, 16, a8, 16, B, c8, 16, D, NULL, E, FP8Q_F32, MAX, NULL), FP8Q_ERR_ALIGN);
  EXPECT(int8_gemm(MAX, 16, 16, a8, 16, B, c8, 16, D, NULL, E, FP8Q_F32, 16, NULL), FP8Q_ERR_UNSUPPORTED);
  EXPECT(int8_gemm(1 << 20, 16, 16, a8, 16, B, c8, 16, D, NULL, E, FP8Q_F32, LD, NULL), FP8Q_ERR_SHAPE);
  EXPECT(int8_gemm(16, 16, MAX, a8, MAX, B, c8, MAX, D, NULL, E, FP8Q_F32, 16, NULL), FP8Q_ERR_ALIGN);
  EXPECT(int8_gemm(16, 16, BIG, a8, BIG, B, c8, BIG, D, NULL, E, FP8Q_F32, 16, NULL), FP8Q_ERR_UNSUPPORTED);
  EXPECT(int8_gemm(16, 16, 17, (const int8_t*)TOP, 32, B, c8, 32, D, NULL, E, FP8Q_F32, 16, NULL), FP8Q_ERR_SHAPE);
  /* the last row is read up to the next multiple of 16 bytes: an output right behind its 17th byte overlaps */
  EXPECT(int8_gemm(2, 16, 17, a8, 32, B, c8, 32, D, NULL, A + 48, FP8Q_F32, 16, NULL), FP8Q_ERR_ALIAS);
  LAUNCHES(int8_gemm(2, 16, 17, a8, 32, B, c8, 32, D, NULL, A + 64, FP8Q_F32, 16, NULL));
  EXPECT(int8_gemm_gated(0, 2, MAX / 2 + 1, 16, a8, 16, B, c8, 16, D, E, FP8Q_F32, MAX, NULL), FP8Q_ERR_SHAPE);
  EXPECT(int8_gemm_gated(0, 2, 16, 131072, a8, 131072, B, c8, 131072, D, E, FP8Q_F32, 16, NULL),
         FP8Q_ERR_UNSUPPORTED);

  if (failures) return 1;
  printf("adversarial validation ok (%d launches reached)\n", fp8q_ffn_stub_launches);
  return 0;
}
