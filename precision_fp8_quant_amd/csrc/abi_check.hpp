// Argument checks shared by the C-ABI layers (host only).
#pragma once

#include "../../include/fp8q.h"

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace {

constexpr int64_t kMaxGridX = 0x7FFFFFFF;
// GEMM operands are read through buffer resources with 32-bit offsets within
// a tile of up to 512 rows: leading dimensions of A and B must stay below
// 2^31 / 512 bytes (4 MiB), with K <= ld.
constexpr int64_t kMaxGemmLd = (int64_t(1) << 31) / 512 - 128;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  uintptr_t lo, hi;   // [lo, hi)
  bool ok;            // false: the extent overflows 64 bits or the address space
};

// Bytes spanned by a row-major matrix with `rows` rows of `cols` elements,
// ((rows - 1) * ld + cols) * esize, with every step checked for overflow
// (the sizes are non-negative here: negative ones were rejected before).
inline Range span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (rows <= 0 || cols <= 0) return {lo, lo, true};
  int64_t elems = 0, bytes = 0;
  uintptr_t hi = 0;
  if (__builtin_mul_overflow(rows - 1, ld, &elems) || __builtin_add_overflow(elems, cols, &elems) ||
      __builtin_mul_overflow(elems, esize, &bytes) || __builtin_add_overflow(lo, uintptr_t(bytes), &hi))
    return {lo, lo, false};
  return {lo, hi, true};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// a * b for non-negative a, b; false on overflow
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

// A leading dimension of `ld` elements of `esize` (2 or 4) bytes is a multiple
// of 16 bytes (without forming ld * esize, which could overflow).
inline bool ld16(int64_t ld, int64_t esize) { return ld % (16 / esize) == 0; }

inline int64_t dtype_size(int dt) { return dt == FP8Q_BF16 ? 2 : 4; }
inline bool dtype_ok(int dt) { return dt == FP8Q_BF16 || dt == FP8Q_F32; }

inline int from_hip(hipError_t e) { return e == hipSuccess ? FP8Q_OK : FP8Q_ERR_HIP; }

}  // namespace
