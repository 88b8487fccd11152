// norm.hpp -- what the norms share (norm.hip, rms.hip): sums over the threads
// of a row, parameters of either type, and the size of a persistent grid.
#pragma once

#include <atomic>

#include "launch.hpp"
#include "rows.hpp"

namespace fp8mi {

// Sums over the NT threads of a row; every thread gets them.  red: two sets of
// one word per wave, used in turn, so one barrier per sum is enough (a set is
// written again only after the barrier of the other).
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (&red)[2][N][16], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[turn][i][wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) s += red[turn][i][w];
      v[i] = s;
    }
    turn ^= 1;
  }
}

template <typename W>
__device__ __forceinline__ void load_param(Chunk<W>& c, const void* p, float otherwise, int col, int n) {
  if (p) c.load(static_cast<const W*>(p) + col, n);
  else c.fill(otherwise);
}

constexpr int threads_of(int nt) { return nt < 256 ? 256 : nt; }

// workgroups of `threads` that stay resident on the stream's device
template <typename Kernel>
int64_t resident(Kernel k, int threads, std::atomic<int>& per_cu_cache, hipStream_t st) {
  int per_cu = per_cu_cache.load(std::memory_order_relaxed);
  if (per_cu <= 0) {
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, k, threads, 0) != hipSuccess || per_cu <= 0) per_cu = 1;
    per_cu_cache.store(per_cu, std::memory_order_relaxed);
  }
  return (int64_t)cu_count(stream_device(st)) * per_cu;
}

}  // namespace fp8mi
