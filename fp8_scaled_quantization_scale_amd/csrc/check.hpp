// check.hpp -- host-side argument checks shared by the C entry points.
#pragma once

#include <stdint.h>

namespace fp8mi {

inline bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// rows x ld elements of esize bytes span a byte range that fits in int64
inline bool span_ok(int64_t rows, int64_t ld, int64_t esize) {
  int64_t n = 0;
  return !__builtin_mul_overflow(rows, ld, &n) && !__builtin_mul_overflow(n, esize, &n);
}

}  // namespace fp8mi
