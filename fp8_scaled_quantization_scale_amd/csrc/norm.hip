// norm.hip -- layer norm over the columns of a BF16 or FP32 matrix, forward
// and backward, for gfx950.
//
//   forward   mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps),
//             y = (x - mu) r w + b
//   backward  h = (x - mu) r, g = dy w,
//             dx = r (g - mean(g) - h mean(g h)),
//             dw = sum over rows of dy h, db = sum over rows of dy
//
// Bound by memory: 2 (forward) or 3 (backward) accesses per element.  A row is
// read once and held in registers by the NT threads that own it (C chunks of
// 8 elements each), so the two passes of the variance cost no second read;
// statistics and sums are FP32.  Workgroups are persistent: the weight (and
// the backward pass's column sums) stay in registers from row to row, and the
// next row's words are on their way while one row is reduced (backward: two
// rows' of 1025 to 8192 columns, one's up to 1024, none's over 8192).
//
// Measured (MI355X): forward 8192 x 16384 BF16 96 us with x partly in the
// caches, 111 without (4.8 TB/s); backward 16384 x 8192 157 us (5.1 TB/s), 8192
// x 4096 45 us (4.5 TB/s).  Over 16384 columns the rows are read again from the
// caches: 4096 x 32768 BF16 forward 171 us (3.1 TB/s), backward 386 (2.1; its
// column sums read x and dy once more), 1024 x 65536 81 (3.3) and 243 (1.7).
//
// The weight's gradient needs a sum over all rows: every workgroup leaves the
// sums of its own rows in a workspace, and a second launch adds these in a
// fixed order, so the result does not depend on which workgroup ends first
// (as it would with atomics).
#include <atomic>

#include "launch.hpp"
#include "rows.hpp"

namespace fp8mi {

namespace {

// Workgroups that leave column sums: each set is 8 bytes per column, written
// and read again, so they are no more than fill the GPU, and each has at least
// 4 rows to add up (1000 x 4000 FP32: 17.7 us; 2 rows 20.2, 1 row 20.3).
constexpr int kMaxPartials = 512;
constexpr int kRowsPerPartial = 4;

struct NormArgs {
  const void* x;
  const void* dy;
  int64_t rows, ld_x, ld_dy, ld_out;
  int cols;
  const void* weight;
  const void* bias;
  float eps;
  float* mean;
  float* rstd;
  void* out;
  float* partial;  // [gridDim.x][2][cols]
};

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

template <typename T, typename W, int NT, int C>
__global__ __launch_bounds__(threads_of(NT)) void norm_forward_kernel(NormArgs a) {
  constexpr int kRows = threads_of(NT) / NT;  // rows per workgroup at a time
  __shared__ float red[2][1][16];
  int turn = 0;
  const int tid = threadIdx.x % NT;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
  const float inv = 1.0f / (float)a.cols;

  int col[C], n[C];
  Chunk<W> w[C], b[C];
  Chunk<T> cur[C], nxt[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * NT + tid) * 8;
    n[c] = a.cols - col[c];  // valid elements of the chunk (may be <= 0)
    if (row < a.rows) cur[c].load(static_cast<const T*>(a.x) + row * a.ld_x + col[c], n[c]);
    load_param(w[c], a.weight, 1.0f, col[c], n[c]);
    load_param(b[c], a.bias, 0.0f, col[c], n[c]);
  }
  for (; row < a.rows; row += step) {
    if (row + step < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) nxt[c].load(static_cast<const T*>(a.x) + (row + step) * a.ld_x + col[c], n[c]);
    }
    float v[C][8], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      cur[c].get(v[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[c][e];  // zeros past the row's end
    }
    row_sum<NT>(s, red, turn);
    const float mean = s[0] * inv;
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[c][e] -= mean;
        s[0] += e < n[c] ? v[c][e] * v[c][e] : 0.0f;
      }
    row_sum<NT>(s, red, turn);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (tid == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float wv[8], bv[8];
      w[c].get(wv);
      b[c].get(bv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = v[c][e] * rstd * wv[e] + bv[e];
      Chunk<T> o;
      o.set(v[c]);
      o.store(static_cast<T*>(a.out) + row * a.ld_out + col[c], n[c]);
      cur[c] = nxt[c];
    }
  }
}

// Rows too long for registers: three passes over each, the later ones from L2.
template <typename T, typename W>
__global__ __launch_bounds__(1024) void norm_forward_long_kernel(NormArgs a) {
  constexpr int NT = 1024;
  __shared__ float red[2][1][16];
  int turn = 0;
  const float inv = 1.0f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    float s[1] = {0.0f};
    for (int col = threadIdx.x * 8; col < a.cols; col += NT * 8) {
      Chunk<T> k;
      float v[8];
      k.load(x + col, a.cols - col);
      k.get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[e];
    }
    row_sum<NT>(s, red, turn);
    const float mean = s[0] * inv;
    s[0] = 0.0f;
    for (int col = threadIdx.x * 8; col < a.cols; col += NT * 8) {
      Chunk<T> k;
      float v[8];
      k.load(x + col, a.cols - col);
      k.get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += e < a.cols - col ? (v[e] - mean) * (v[e] - mean) : 0.0f;
    }
    row_sum<NT>(s, red, turn);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    for (int col = threadIdx.x * 8; col < a.cols; col += NT * 8) {
      Chunk<T> k;
      Chunk<W> w, b;
      float v[8], wv[8], bv[8];
      k.load(x + col, a.cols - col);
      load_param(w, a.weight, 1.0f, col, a.cols - col);
      load_param(b, a.bias, 0.0f, col, a.cols - col);
      k.get(v);
      w.get(wv);
      b.get(bv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (v[e] - mean) * rstd * wv[e] + bv[e];
      k.set(v);
      k.store(static_cast<T*>(a.out) + row * a.ld_out + col, a.cols - col);
    }
  }
}

template <typename T, typename W, int NT, int C, int AHEAD>
__global__ __launch_bounds__(threads_of(NT)) void norm_backward_kernel(NormArgs a) {
  constexpr int kRows = threads_of(NT) / NT;
  __shared__ float red[2][2][16];
  int turn = 0;
  const int tid = threadIdx.x % NT;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
  const float inv = 1.0f / (float)a.cols;

  constexpr int kAhead = AHEAD;  // rows on their way beside the one in hand
  int col[C], n[C];
  Chunk<W> w[C];
  Chunk<T> cx[kAhead + 1][C], cy[kAhead + 1][C];
  float mean[kAhead + 1], rstd[kAhead + 1];
  float dw[C][8], db[C][8];
  auto fetch = [&](int q, int64_t r) __attribute__((always_inline)) {
    if (r < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        cx[q][c].load(static_cast<const T*>(a.x) + r * a.ld_x + col[c], n[c]);
        cy[q][c].load(static_cast<const T*>(a.dy) + r * a.ld_dy + col[c], n[c]);
      }
      mean[q] = a.mean[r];
      rstd[q] = a.rstd[r];
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * NT + tid) * 8;
    n[c] = a.cols - col[c];
  }
#pragma unroll
  for (int q = 0; q < kAhead; ++q) fetch(q, row + q * step);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_param(w[c], a.weight, 1.0f, col[c], n[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = db[c][e] = 0.0f;
  }
  for (; row < a.rows; row += step) {
    fetch(kAhead, row + kAhead * step);
    float s[2] = {0.0f, 0.0f};  // sums of g and g h (dy is zero past the row's end)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float x[8], y[8], wv[8];
      cx[0][c].get(x);
      cy[0][c].get(y);
      w[c].get(wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = (x[e] - mean[0]) * rstd[0], g = y[e] * wv[e];
        s[0] += g;
        s[1] += g * h;
        dw[c][e] += y[e] * h;
        db[c][e] += y[e];
      }
    }
    row_sum<NT>(s, red, turn);
    const float m1 = s[0] * inv, m2 = s[1] * inv;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float x[8], y[8], wv[8], o[8];
      cx[0][c].get(x);
      cy[0][c].get(y);
      w[c].get(wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = (x[e] - mean[0]) * rstd[0], g = y[e] * wv[e];
        o[e] = rstd[0] * (g - m1 - h * m2);
      }
      Chunk<T> k;
      k.set(o);
      k.store(static_cast<T*>(a.out) + row * a.ld_out + col[c], n[c]);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        cx[q][c] = cx[q + 1][c];
        cy[q][c] = cy[q + 1][c];
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      mean[q] = mean[q + 1];
      rstd[q] = rstd[q + 1];
    }
  }
  if (!a.partial) return;
  float* p = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      Chunk<float> k;
      k.set(dw[c]);
      k.store(p + col[c], n[c]);
      k.set(db[c]);
      k.store(p + a.cols + col[c], n[c]);
    }
  } else {
    // the workgroup's rows side by side: added here, in order
    __shared__ float sums[kRows][2][C * NT * 8];
    const int g = threadIdx.x / NT;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[g][0][col[c] + e] = dw[c][e];
        sums[g][1][col[c] + e] = db[c][e];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.cols; i += threads_of(NT)) {
      const int k = i >= a.cols, j = i - k * a.cols;
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += sums[r][k][j];
      p[i] = s;
    }
  }
}

// Rows too long for registers: dx only, two passes over each row.
template <typename T, typename W>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(NormArgs a) {
  constexpr int NT = 1024;
  __shared__ float red[2][2][16];
  int turn = 0;
  const float inv = 1.0f / (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* yr = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.0f, 0.0f};
    for (int pass = 0; pass < 2; ++pass) {
      for (int col = threadIdx.x * 8; col < a.cols; col += NT * 8) {
        Chunk<T> kx, ky;
        Chunk<W> kw;
        float x[8], y[8], w[8], o[8];
        kx.load(xr + col, a.cols - col);
        ky.load(yr + col, a.cols - col);
        load_param(kw, a.weight, 1.0f, col, a.cols - col);
        kx.get(x);
        ky.get(y);
        kw.get(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float h = (x[e] - mean) * rstd, g = y[e] * w[e];
          if (pass == 0) {
            s[0] += g;
            s[1] += g * h;
          }
          o[e] = rstd * (g - s[0] - h * s[1]);
        }
        if (pass == 1) {
          kx.set(o);
          kx.store(static_cast<T*>(a.out) + row * a.ld_out + col, a.cols - col);
        }
      }
      if (pass == 0) {
        row_sum<NT>(s, red, turn);
        s[0] *= inv;
        s[1] *= inv;
      }
    }
  }
}

// ... and their column sums: a wave owns 512 columns of gridDim.y-strided rows.
template <typename T>
__global__ __launch_bounds__(64) void norm_columns_kernel(NormArgs a) {
  const int col = ((int)blockIdx.x * 64 + threadIdx.x) * 8, n = a.cols - col;
  if (n <= 0) return;
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    Chunk<T> kx, ky;
    float x[8], y[8];
    kx.load(static_cast<const T*>(a.x) + row * a.ld_x + col, n);
    ky.load(static_cast<const T*>(a.dy) + row * a.ld_dy + col, n);
    kx.get(x);
    ky.get(y);
    const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e] += y[e] * ((x[e] - mean) * rstd);
      db[e] += y[e];
    }
  }
  float* p = a.partial + (int64_t)blockIdx.y * 2 * a.cols;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) {
      p[col + e] = dw[e];
      p[a.cols + col + e] = db[e];
    }
}

// dw and db from the workgroups' sums: a workgroup takes 32 of the 2 cols
// columns, four to a thread, and each of its 128 thread groups every 128th
// partial, so that even a short norm's sums are read by many compute units.
// A launch has its work-items counted modulo 2^32, and a column takes 64 of
// them: from 2^26 columns on there are several launches, each with its first
// group.
constexpr int kReduceCols = 32, kReduceGroups = 128;
constexpr int64_t kReduceMost = (1LL << 31) / 1024;  // workgroups of a launch
template <typename W>
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* partial, int parts, int cols, W* dw, W* db,
                                                           int64_t first) {
  __shared__ float sums[kReduceGroups][kReduceCols + 4];
  const int64_t width = 2 * (int64_t)cols;
  const int at = (threadIdx.x & 7) * 4, group = threadIdx.x >> 3;
  const int64_t i = (first + blockIdx.x) * kReduceCols + at;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i + 4 <= width) {
    for (int p = group; p < parts; p += kReduceGroups) {
      const f32x4a4 v = *reinterpret_cast<const f32x4a4*>(partial + p * width + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
  } else {
    for (int p = group; p < parts; p += kReduceGroups)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < width) s[e] += partial[p * width + i + e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[group][at + e] = s[e];
  __syncthreads();
  // 32 threads per column, then one
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < kReduceGroups / 32; ++k) q += sums[g * (kReduceGroups / 32) + k][c];
  __syncthreads();
  sums[g][c] = q;
  __syncthreads();
  const int64_t j = (first + blockIdx.x) * kReduceCols + c;
  if (g != 0 || j >= width) return;
  q = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) q += sums[k][c];
  W* dst = j < cols ? dw : db;
  if (!dst) return;
  const int64_t to = j < cols ? j : j - cols;
  if constexpr (sizeof(W) == 4) dst[to] = q;
  else dst[to] = __builtin_bit_cast(uint16_t, (__bf16)q);
}

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

NormArgs args_of(const NormParams& p) {
  return NormArgs{p.x,      p.dy,   p.rows, p.ld_x, p.ld_dy, p.ld_out, (int)p.cols, p.weight,
                  p.bias, p.eps, p.mean,  p.rstd, p.out,  nullptr};
}

template <typename T, typename W, int NT, int C>
hipError_t forward(const NormParams& p, hipStream_t st) {
  static std::atomic<int> occupancy{0};
  auto k = norm_forward_kernel<T, W, NT, C>;
  constexpr int threads = threads_of(NT), rows = threads / NT;
  const int64_t need = (p.rows + rows - 1) / rows, most = resident(k, threads, occupancy, st);
  k<<<(unsigned)(need < most ? need : most), threads, 0, st>>>(args_of(p));
  return hipGetLastError();
}

template <typename T, typename W>
hipError_t forward_any(const NormParams& p, hipStream_t st) {
  if (p.cols <= 512) return forward<T, W, 64, 1>(p, st);
  if (p.cols <= 1024) return forward<T, W, 64, 2>(p, st);
  if (p.cols <= 2048) return forward<T, W, 256, 1>(p, st);
  if (p.cols <= 4096) return forward<T, W, 256, 2>(p, st);
  if (p.cols <= 8192) return forward<T, W, 512, 2>(p, st);
  if (p.cols <= 16384) return forward<T, W, 1024, 2>(p, st);
  const int64_t most = 2 * (int64_t)cu_count(stream_device(st));
  norm_forward_long_kernel<T, W><<<(unsigned)(p.rows < most ? p.rows : most), 1024, 0, st>>>(args_of(p));
  return hipGetLastError();
}

template <typename W>
hipError_t reduce(const NormParams& p, int parts, hipStream_t st) {
  if (!p.dweight && !p.dbias) return hipGetLastError();
  const int64_t groups = (2 * p.cols + kReduceCols - 1) / kReduceCols;
  for (int64_t g = 0; g < groups; g += kReduceMost) {
    const int64_t n = groups - g < kReduceMost ? groups - g : kReduceMost;
    norm_reduce_kernel<W><<<(unsigned)n, 1024, 0, st>>>(p.workspace, parts, (int)p.cols, static_cast<W*>(p.dweight),
                                                        static_cast<W*>(p.dbias), g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, typename W, int NT, int C, int AHEAD>
hipError_t backward(const NormParams& p, hipStream_t st) {
  static std::atomic<int> occupancy{0};
  auto k = norm_backward_kernel<T, W, NT, C, AHEAD>;
  constexpr int threads = threads_of(NT);
  int64_t blocks = norm_partials(p.rows);
  const int64_t most = resident(k, threads, occupancy, st);
  blocks = blocks < most ? blocks : most;
  NormArgs a = args_of(p);
  a.partial = p.dweight || p.dbias ? p.workspace : nullptr;
  if (p.rows > 0) {
    k<<<(unsigned)blocks, threads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return reduce<W>(p, p.rows > 0 ? (int)blocks : 0, st);
}

template <typename T, typename W>
hipError_t backward_any(const NormParams& p, hipStream_t st) {
  // Threads and chunks per row: few enough threads that a row's sum ends in
  // few waves, few enough chunks that sums, weight and the rows ahead stay in
  // registers.  Two rows ahead beat one where they fit (8192 x 4096 BF16: 42 us
  // against 47); a 16384-column row leaves no room for any (8192 rows BF16: 165
  // us, with 2 registers spilled, 6 beside FP32 weights; one row ahead 275 us of
  // spills; 512 threads of 4 chunks 162 us).
  if (p.cols <= 512) return backward<T, W, 64, 1, 1>(p, st);
  if (p.cols <= 1024) return backward<T, W, 64, 2, 1>(p, st);
  if (p.cols <= 2048) return backward<T, W, 256, 1, 2>(p, st);
  if (p.cols <= 4096) return backward<T, W, 256, 2, 2>(p, st);
  if (p.cols <= 8192) return backward<T, W, 512, 2, 2>(p, st);
  if (p.cols <= 16384) return backward<T, W, 1024, 2, 0>(p, st);
  if (p.rows == 0) return reduce<W>(p, 0, st);
  const int64_t most = 2 * (int64_t)cu_count(stream_device(st));
  NormArgs a = args_of(p);
  norm_backward_long_kernel<T, W><<<(unsigned)(p.rows < most ? p.rows : most), 1024, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
  a.partial = p.workspace;
  const int64_t parts = norm_partials(p.rows);
  norm_columns_kernel<T><<<dim3((unsigned)((p.cols + 511) / 512), (unsigned)parts), 64, 0, st>>>(a);
  e = hipGetLastError();
  return e != hipSuccess ? e : reduce<W>(p, (int)parts, st);
}

}  // namespace

// sets of column sums that a backward pass over `rows` rows may leave
int64_t norm_partials(int64_t rows) {
  const int64_t n = (rows + kRowsPerPartial - 1) / kRowsPerPartial;
  return n < 1 ? 1 : (n < kMaxPartials ? n : kMaxPartials);
}

hipError_t launch_norm_forward(const NormParams& p, hipStream_t st) {
  if (p.rows == 0) return hipSuccess;
  if (p.x_dtype == kInBf16)
    return p.w_dtype == kInBf16 ? forward_any<uint16_t, uint16_t>(p, st) : forward_any<uint16_t, float>(p, st);
  return p.w_dtype == kInBf16 ? forward_any<float, uint16_t>(p, st) : forward_any<float, float>(p, st);
}

hipError_t launch_norm_backward(const NormParams& p, hipStream_t st) {
  if (p.x_dtype == kInBf16)
    return p.w_dtype == kInBf16 ? backward_any<uint16_t, uint16_t>(p, st) : backward_any<uint16_t, float>(p, st);
  return p.w_dtype == kInBf16 ? backward_any<float, uint16_t>(p, st) : backward_any<float, float>(p, st);
}

}  // namespace fp8mi
