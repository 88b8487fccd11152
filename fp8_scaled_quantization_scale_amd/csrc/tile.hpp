// tile.hpp -- pieces of the kernels that leave FP8 codes, on 128 x 128 tiles or
// by the row: block maxima over the lanes that share a block, the encoders and
// their stores (quantize.hip, rms.hip).
#pragma once

#include <type_traits>

#include "device.hpp"

namespace fp8mi {

constexpr int kTile = 128;
// byte stride of the transposed code tile staged in LDS: 144 = 128 + 16 keeps
// 16-byte alignment and spreads the column writes of a wave over the banks
constexpr int kCodeStride = 144;

// ROW codes are written whole-line by consecutive lanes and not read again
// by this pass, so they are stored non-temporally (measured on MI355X: an
// 8192x4096 ROW cast 20.9 -> 18.6 us).  Non-temporal loads of the input and
// non-temporal COL stores measured slower.
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st_stream8(void* p, uint2 w) {
  const u32x2_t v = {w.x, w.y};
  __builtin_nontemporal_store(v, reinterpret_cast<u32x2_t*>(p));
}

enum : int { MODE_TENSOR = 0, MODE_B1x128 = 1, MODE_B128x128 = 2, MODE_MX32 = 3, MODE_CHANNEL = 4, MODE_MX32F = 5 };

// E8M0 byte of an MX block: MODE_MX32 takes the smallest power of two under
// which no element saturates, MODE_MX32F the OCP specification's floor rule.
template <int MODE, int FMT>
__device__ __forceinline__ int mx_byte(float amax) {
  if constexpr (MODE == MODE_MX32F) return mx_scale_byte_floor<FMT>(amax);
  else return mx_scale_byte<FMT>(amax);
}

template <int FMT, bool Safe>
__device__ __forceinline__ uint2 encode8(const float v[8], float s) {
  uint2 r;
  r.x = encode4<FMT, Safe>(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
  r.y = encode4<FMT, Safe>(v[4] * s, v[5] * s, v[6] * s, v[7] * s);
  return r;
}

__device__ __forceinline__ void store8(uint8_t* q, int64_t n, uint2 c) {
  if (n >= 8) {
    st_stream8(q, c);
  } else {
    for (int e = 0; e < n; ++e) q[e] = (uint8_t)((e < 4 ? c.x >> (8 * e) : c.y >> (8 * (e - 4))) & 0xFF);
  }
}

__device__ __forceinline__ uint32_t max8_key(const float v[8]) {
  uint32_t k = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t t = abs_key(v[e]);
    k = k > t ? k : t;
  }
  return k;
}

// Delayed scaling: the convert-only encoder is exact for a chunk whose
// largest magnitude m is finite with fl32(m * s) <= max (every product then
// rounds to at most max); anything else takes the saturating encoder.
template <int FMT>
__device__ __forceinline__ bool fits(uint32_t key, float s) {
  const float m = key_to_float(key);
  return m <= kFltMax && m * s <= Fmt<FMT>::kMax;
}

// max |x| key of 8 BF16 values packed in a uint4: packed 16-bit max of the
// sign-cleared halves (non-negative BF16 orders like its bits, NaN on top).
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x8_key(uint4 w) {
  u16x2 m = __builtin_bit_cast(u16x2, w.x & 0x7FFF7FFFu);
  m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.y & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.z & 0x7FFF7FFFu));
  m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w.w & 0x7FFF7FFFu));
  const uint32_t k = m.x > m.y ? m.x : m.y;
  return k << 16;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }
// max over the 16 lanes of a DPP row (rotations) / over 4 lanes (quad permutes)
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = umax32(v, dpp<0x128>(v));
  v = umax32(v, dpp<0x124>(v));
  v = umax32(v, dpp<0x122>(v));
  return umax32(v, dpp<0x121>(v));
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = umax32(v, dpp<0x4E>(v));         // lanes 2 3 0 1
  return umax32(v, dpp<0xB1>(v));      // lanes 1 0 3 2
}
// lane N of every row of 16, to all of that row
template <int N>
__device__ __forceinline__ float row16_lane(float v) {
  return __builtin_bit_cast(float, dpp<0x150 + N>(__builtin_bit_cast(uint32_t, v)));
}

// sum over a row of 16 lanes, to all of them, by rotations
__device__ __forceinline__ float row16_total(float v) {
  v += __builtin_bit_cast(float, dpp<0x128>(__builtin_bit_cast(uint32_t, v)));
  v += __builtin_bit_cast(float, dpp<0x124>(__builtin_bit_cast(uint32_t, v)));
  v += __builtin_bit_cast(float, dpp<0x122>(__builtin_bit_cast(uint32_t, v)));
  return v + __builtin_bit_cast(float, dpp<0x121>(__builtin_bit_cast(uint32_t, v)));
}

// sum over the 64 lanes of a wave, to all of them: the rows' sums as scalars
__device__ __forceinline__ float wave_total(float v) {
  v = row16_total(v);
  auto row = [&](int lane) __attribute__((always_inline)) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  };
  return (row(0) + row(16)) + (row(32) + row(48));
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }

template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (N > 0) {
    unrolled<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

}  // namespace fp8mi
