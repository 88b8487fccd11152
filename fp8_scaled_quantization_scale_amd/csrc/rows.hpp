// rows.hpp -- 8 consecutive elements of a BF16 or FP32 row, for the kernels
// that work on whole rows (layer norm, expert dispatch and combine).
//
// Rows may start at any element: an 8-element chunk is moved as 16-byte words
// whatever its address (gfx950 takes dword and larger global accesses at any
// byte address), and only the chunk that a row's end cuts goes element by
// element.
#pragma once

#include "device.hpp"

namespace fp8mi {

typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

// NT: written past the caches, for output that nothing reads before it would
// have left them anyway.  (Not a template over the vector's type: deduction
// drops the typedefs' alignment, and the stores would claim 16 bytes.)
template <bool NT>
__device__ __forceinline__ void put(u32x4a2 v, u32x4a2* p) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool NT>
__device__ __forceinline__ void put(f32x4a4 v, f32x4a4* p) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// the 8 elements as they lie in memory (BF16: 16 bytes, FP32: 32)
template <typename T>
struct Chunk;

template <>
struct Chunk<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p, int64_t n) {
    if (n >= 8) {
      const u32x4a2 v = *reinterpret_cast<const u32x4a2*>(p);
      w = make_uint4(v.x, v.y, v.z, v.w);
    } else {
      uint32_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) h[e] = p[e];
      w = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    }
  }
  __device__ __forceinline__ void fill(float v) {
    const uint32_t h = __builtin_bit_cast(uint32_t, v) >> 16, p = h | (h << 16);
    w = make_uint4(p, p, p, p);
  }
  __device__ __forceinline__ void get(float v[8]) const { unpack_bf16x8(w, v); }
  // nearest-even
  __device__ __forceinline__ void set(const float v[8]) {
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __bf16 lo = (__bf16)v[2 * e], hi = (__bf16)v[2 * e + 1];
      p[e] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
    }
    w = make_uint4(p[0], p[1], p[2], p[3]);
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(uint16_t* p, int64_t n) const {
    if (n >= 8) {
      const u32x4a2 v = {w.x, w.y, w.z, w.w};
      put<NT>(v, reinterpret_cast<u32x4a2*>(p));
    } else {
      const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
    }
  }
};

template <>
struct Chunk<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float* p, int64_t n) {
    if (n >= 8) {
      const f32x4a4 a = reinterpret_cast<const f32x4a4*>(p)[0], b = reinterpret_cast<const f32x4a4*>(p)[1];
      lo = make_float4(a.x, a.y, a.z, a.w);
      hi = make_float4(b.x, b.y, b.z, b.w);
    } else {
      lo.x = n > 0 ? p[0] : 0.0f;
      lo.y = n > 1 ? p[1] : 0.0f;
      lo.z = n > 2 ? p[2] : 0.0f;
      lo.w = n > 3 ? p[3] : 0.0f;
      hi.x = n > 4 ? p[4] : 0.0f;
      hi.y = n > 5 ? p[5] : 0.0f;
      hi.z = n > 6 ? p[6] : 0.0f;
      hi.w = 0.0f;
    }
  }
  __device__ __forceinline__ void fill(float v) { lo = hi = make_float4(v, v, v, v); }
  __device__ __forceinline__ void get(float v[8]) const {
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
  __device__ __forceinline__ void set(const float v[8]) {
    lo = make_float4(v[0], v[1], v[2], v[3]);
    hi = make_float4(v[4], v[5], v[6], v[7]);
  }
  template <bool NT = false>
  __device__ __forceinline__ void store(float* p, int64_t n) const {
    if (n >= 8) {
      put<NT>(f32x4a4{lo.x, lo.y, lo.z, lo.w}, reinterpret_cast<f32x4a4*>(p));
      put<NT>(f32x4a4{hi.x, hi.y, hi.z, hi.w}, reinterpret_cast<f32x4a4*>(p) + 1);
    } else {
      if (n > 0) p[0] = lo.x;
      if (n > 1) p[1] = lo.y;
      if (n > 2) p[2] = lo.z;
      if (n > 3) p[3] = lo.w;
      if (n > 4) p[4] = hi.x;
      if (n > 5) p[5] = hi.y;
      if (n > 6) p[6] = hi.z;
    }
  }
};

// Sum over the 64 lanes of a wave; every lane gets it.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

}  // namespace fp8mi
