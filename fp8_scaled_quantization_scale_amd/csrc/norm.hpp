// norm.hpp -- what the norms share (norm.hip, rms.hip): the size of a workgroup
// and of a persistent grid.
#pragma once

#include <atomic>

#include "launch.hpp"
#include "rows.hpp"

namespace fp8mi {

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
