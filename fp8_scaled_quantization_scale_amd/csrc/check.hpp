// check.hpp -- host-side argument checks shared by the C entry points.
#pragma once

#include <stdint.h>

#include "fp8mi.h"

namespace fp8mi {

inline bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// rows x ld elements of esize bytes span a byte range that fits in int64 (no
// array that large can exist; checking first keeps every later size
// computation here and in the launchers free of overflow)
inline bool span_ok(int64_t rows, int64_t ld, int64_t esize) {
  int64_t n = 0;
  return !__builtin_mul_overflow(rows, ld, &n) && !__builtin_mul_overflow(n, esize, &n);
}

// BF16 and FP32 inputs
inline bool in_dtype_ok(int d) { return d == FP8MI_IN_BF16 || d == FP8MI_IN_FP32; }
inline int64_t in_size(int d) { return d == FP8MI_IN_BF16 ? 2 : 4; }

// a row-major matrix whose pointer is aligned to its elements
inline int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
  if (!p) return FP8MI_ERR_NULL;
  if (ld < cols || !span_ok(rows, ld, esize)) return FP8MI_ERR_SHAPE;
  return aligned_to(p, esize) ? FP8MI_OK : FP8MI_ERR_ALIGN;
}

}  // namespace fp8mi
