// rms.hip -- root-mean-square norm over the columns of a BF16 or FP32 matrix,
// with the addition of a residual before it, forward (to the matrix's type or
// straight to FP8 codes) and backward, for gfx950.
//
//   forward   t = x + residual, rounded to its type,
//             r = 1 / sqrt(mean(t^2) + eps), y = t r w
//   backward  n = t r, g = dy w,
//             dx = r (g - n mean(g n)) + dt   (dt: the gradient that reaches t
//             by itself, along the residual stream; dx is the residual's too),
//             dw = sum over rows of dy n
//
// Bound by memory.  As in the layer norm a row is read once and held in
// registers by the NT threads that own it (C chunks of 8 elements each),
// workgroups are persistent, and the next row's words are on their way while
// one row is reduced.  y is worked out in FP32, t r first and then w, and rounded
// once: for codes too, whose scales are those of the FP32 y.
//
// Codes with their blocks along the columns (ROW) leave from the same
// registers: a 1x128 block is 16 neighbouring lanes' chunks, an MX block four
// lanes'.  Codes with their blocks along the rows (COL) need 128 rows'
// statistics before their first element, so a second launch reads t again, in
// 128 x 128 tiles.  (Rows in parts of 128, 64 or 32 MB of t, each with both launches
// and its inputs read past the caches, so that t would still be in the Infinity
// Cache: 8192 x 16384 takes 240, 262 or 295 us against 240 in one part; what the
// cache gives goes to the launches' ends.)
//
// Measured (MI355X, BF16 with a residual): forward 8192 x 16384 183 us (5.9
// TB/s); into 1x128 codes of both orientations 156 + 79 us (5.8 TB/s of the 1.37
// GB that the two launches move), 8192 x 4096 42 + 19 us, under delayed scaling 60 in
// all; backward 8192 x 4096 46 us (6.0 TB/s) and 4.7 of the weight's sums, 4096 x
// 16384 102 us in all (5.2 TB/s).  Over 16384 columns the rows are read again from
// the caches.
#include "norm.hpp"
#include "tile.hpp"

namespace fp8mi {

namespace {

// Workgroups that leave column sums: each set is 4 bytes per column, written and
// read again, so they are no more than fill the GPU, and each has as many rows at
// least as it takes at a time: 16 of up to 256 columns, 4 of up to 1024, else one.
// There it takes 4 too, fewer where that leaves compute units without work (64 x
// 2560: 1 row 6.4 us, 4 10.2; 256 x 4096: 1 8.5, 2 8.1, 4 9.6; 512 x 4096: 13.3,
// 11.3, 11.6).  The sums of the short rows are so few that twice as many sets cost
// little (BF16, 512 or 1024 sets: 262144 x 64 41 or 29 us, 262144 x 128 44 or 41,
// 65536 x 256 26.9 or 28.4; wider rows lose, 65536 x 1024 94 or 100).
constexpr int64_t kMaxPartials = 512, kMaxShortPartials = 1024;
constexpr int64_t kShort = 256, kMiddle = 1024;  // columns
constexpr int64_t rows_per_partial(int64_t rows, int64_t cols) {
  if (cols <= kShort) return 16;
  return cols <= kMiddle || rows > 1024 ? 4 : (rows <= 128 ? 1 : 2);
}

struct RmsArgs {
  const void* x;         // backward: t
  const void* residual;  // backward: dt
  const void* dy;
  int64_t rows, ld_x, ld_residual, ld_dy, ld_total, ld_out;
  int cols;
  double inv;  // 1 / cols
  const void* weight;
  int w_bf16;
  float eps;
  void* total;
  void* out;  // y or dx (nullptr: neither)
  float* rstd;
  float* partial;  // [gridDim.x][cols]
  // codes
  uint8_t* q;
  void* scales;
  int64_t ld_q;
  int margin, floor_rule;
  int32_t* nonfinite;
  const float* scale;  // delayed: the tensor's, and a slot of |y|'s maximum per workgroup
  uint32_t* amax;
};

// sum of N numbers, a power of two, in pairs
template <int N, typename S>
__device__ __forceinline__ S paired_sum(const float* v) {
  if constexpr (N == 1) return v[0];
  else return paired_sum<N / 2, S>(v) + paired_sum<N / 2, S>(v + N / 2);
}

// Sum over the NT threads of a row, to all of them, the waves' sums in 64 bits (one
// after the other in FP32 they cost rstd a fifth of its error at 16384 columns; no
// time in either form).  red: two sets of one word
// per wave, used in turn, so that one barrier is enough (a set is written again
// only after the barrier of the other).  Within a wave by rotations (four rows to
// a wave for NT = 16), whose latency is a fraction of the shuffles' (128 x 512
// forward 2.9 us by shuffles, 2.6 by rotations; 8192 x 5120 backward 89.0, 85.6).
// SHUFFLE is the backward pass over FP32 rows of 2049 to 4096 columns, the one place
// where shuffles measured faster (1000 x 4000 15.3 us, rotations 16.3; 2000 x 4000
// 27.4, 29.6; 4096 x 4096 48.8, 50.1; 8192 x 4096 alike), with one workgroup to a
// compute unit: its 132 VGPRs are four too many for two.
template <int NT, bool SHUFFLE = false>
__device__ __forceinline__ double sum_of_row(float v, float (&red)[2][16], int& turn) {
  if constexpr (NT == 16) v = row16_total(v);
  else if constexpr (SHUFFLE) v = wave_sum(v);
  else v = wave_total(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    turn ^= 1;
    return paired_sum<NT / 64, double>(red[turn ^ 1]);
  }
  return v;
}

// v / cols, rounded once
__device__ __forceinline__ float mean_of(double v, double inv) { return (float)(v * inv); }

// Sums of squares: eight partial sums, so that few roundings follow one another
struct Squares {
  float s[8] = {};
  __device__ __forceinline__ void add(const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += v[e] * v[e];
  }
  __device__ __forceinline__ float total() const { return paired_sum<8, float>(s); }
};

enum : int { OUT_VALUES = 0, OUT_BLOCK = 1, OUT_MX = 2, OUT_TENSOR = 3 };  // what a forward kernel leaves

// 8 weights as floats (1 without one; 0 past the end)
__device__ __forceinline__ void load_weight(float (&v)[8], const RmsArgs& a, int col, int n) {
  if (!a.weight) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
  } else if (a.w_bf16) {
    Chunk<uint16_t> c;
    c.load(static_cast<const uint16_t*>(a.weight) + col, n);
    c.get(v);
  } else {
    Chunk<float> c;
    c.load(static_cast<const float*>(a.weight) + col, n);
    c.get(v);
  }
}

// Codes and scale of a lane's 8 elements of row `row` from column `col` on, n
// of them in the row (zeros past its end); every lane of the block calls it.
// `s` and `most`: the tensor's scale and the largest |y| so far (OUT_TENSOR).
template <int OUT, int FMT>
__device__ __forceinline__ void put_codes(const RmsArgs& a, int64_t row, int col, int n, const float (&y)[8], float s,
                                          uint32_t& most) {
  uint32_t key = max8_key(y);
  bool safe;
  if constexpr (OUT == OUT_TENSOR) {
    if (n > 0) most = umax32(most, key);
    safe = !fits<FMT>(key, s);
    if (!a.q) return;
  } else if constexpr (OUT == OUT_BLOCK) {
    key = row16_max(key);
    const float am = key_to_float(key);
    s = scale_from_amax<FMT>(am, a.margin);
    safe = !is_finite(am);
    if ((threadIdx.x & 15) == 0 && n > 0) {
      const int blocks = (a.cols + 127) / 128;
      static_cast<float*>(a.scales)[row * blocks + (col >> 7)] = recip_rn(s);
      if (safe && a.nonfinite) atomicAdd(a.nonfinite, 1);
    }
  } else {
    key = quad_max(key);
    const float am = key_to_float(key);
    const int byte = a.floor_rule ? mx_scale_byte_floor<FMT>(am) : mx_scale_byte<FMT>(am);
    s = byte == 0xFF ? 1.0f : mx_inv_scale(byte);
    safe = byte == 0xFF || a.floor_rule;
    if ((threadIdx.x & 3) == 0 && n > 0) {
      const int blocks = (a.cols + 31) / 32;
      static_cast<uint8_t*>(a.scales)[row * blocks + (col >> 5)] = (uint8_t)byte;
      if (byte == 0xFF && a.nonfinite) atomicAdd(a.nonfinite, 1);
    }
  }
  if (n > 0) store8(a.q + row * a.ld_q + col, n, safe ? encode8<FMT, true>(y, s) : encode8<FMT, false>(y, s));
}

// OUT_TENSOR: the workgroup's largest |y| into its slot (one workgroup's alone:
// the grid is no more than there are slots), beside what is there.
__device__ __forceinline__ void put_amax(const RmsArgs& a, uint32_t most) {
  __shared__ uint32_t red[16];
  most = group_max_u32<64>(most);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (unsigned w = 1; w < blockDim.x / 64; ++w) most = umax32(most, red[w]);
    a.amax[blockIdx.x] = umax32(a.amax[blockIdx.x], most);
  }
}

// PAST: read and written past the caches.  AGAIN: t is read again by the launch that
// follows (COL codes), so it is written as usual; OUT_VALUES then leaves t and rstd
// alone, for COL codes without ROW ones.
template <typename T, int NT, int C, int OUT, int FMT, bool PAST, bool AGAIN>
__global__ __launch_bounds__(threads_of(NT)) void rms_forward_kernel(RmsArgs a) {
  constexpr int kRows = threads_of(NT) / NT;  // rows per workgroup at a time
  __shared__ float red[2][16];
  int turn = 0;
  const int tid = threadIdx.x % NT;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;

  int col[C], n[C];
  float w[C][8];
  const float scale = OUT == OUT_TENSOR ? *a.scale : 1.0f;
  uint32_t most = 0;
  Chunk<T> cx[C], cr[C], nx[C], nr[C];
  auto fetch = [&](Chunk<T>(&x)[C], Chunk<T>(&r)[C], int64_t at) __attribute__((always_inline)) {
    if (at < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        x[c].template load<PAST>(static_cast<const T*>(a.x) + at * a.ld_x + col[c], n[c]);
        if (a.residual) r[c].template load<PAST>(static_cast<const T*>(a.residual) + at * a.ld_residual + col[c], n[c]);
      }
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * NT + tid) * 8;
    n[c] = a.cols - col[c];  // valid elements of the chunk (may be <= 0)
  }
  fetch(cx, cr, row);
#pragma unroll
  for (int c = 0; c < C; ++c) load_weight(w[c], a, col[c], n[c]);
  for (; row < a.rows; row += step) {
    fetch(nx, nr, row + step);
    float v[C][8];
    Squares squares;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      cx[c].get(v[c]);
      if (a.residual) {
        float r[8];
        cr[c].get(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] += r[e];
        cx[c].set(v[c]);
        cx[c].template store<PAST && !AGAIN>(static_cast<T*>(a.total) + row * a.ld_total + col[c], n[c]);
        cx[c].get(v[c]);
      }
      squares.add(v[c]);  // zeros past the row's end
    }
    const double s = sum_of_row<NT>(squares.total(), red, turn);
    const float rstd = 1.0f / sqrtf(mean_of(s, a.inv) + a.eps);
    if (tid == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = v[c][e] * rstd * w[c][e];
      if constexpr (OUT == OUT_VALUES) {
        if (!AGAIN) {
          Chunk<T> o;
          o.set(v[c]);
          o.template store<PAST>(static_cast<T*>(a.out) + row * a.ld_out + col[c], n[c]);
        }
      } else {
        put_codes<OUT, FMT>(a, row, col[c], n[c], v[c], scale, most);
      }
      cx[c] = nx[c];
      cr[c] = nr[c];
    }
  }
  if constexpr (OUT == OUT_TENSOR) put_amax(a, most);
}

// Rows too long for registers: a second pass over each, from the caches.
template <typename T, int OUT, int FMT>
__global__ __launch_bounds__(1024) void rms_forward_long_kernel(RmsArgs a) {
  constexpr int NT = 1024;
  __shared__ float red[2][16];
  int turn = 0;
  const float scale = OUT == OUT_TENSOR ? *a.scale : 1.0f;
  uint32_t most = 0;
  // (whole turns of the workgroup: the lanes of a block go together)
  const int end = (a.cols + NT * 8 - 1) / (NT * 8) * (NT * 8);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    T* t = static_cast<T*>(a.total) + row * a.ld_total;
    Squares squares;
    for (int col = threadIdx.x * 8; col < a.cols; col += NT * 8) {
      Chunk<T> k;
      float v[8];
      k.load(x + col, a.cols - col);
      k.get(v);
      if (a.residual) {
        float r[8];
        k.load(static_cast<const T*>(a.residual) + row * a.ld_residual + col, a.cols - col);
        k.get(r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += r[e];
        k.set(v);
        k.store(t + col, a.cols - col);
        k.get(v);
      }
      squares.add(v);
    }
    const double s = sum_of_row<NT>(squares.total(), red, turn);
    const float rstd = 1.0f / sqrtf(mean_of(s, a.inv) + a.eps);
    if (threadIdx.x == 0) a.rstd[row] = rstd;
    if (OUT == OUT_VALUES && !a.out) continue;
    if (a.residual) x = t;  // (each thread reads what it wrote)
    for (int col = threadIdx.x * 8; col < end; col += NT * 8) {
      Chunk<T> k;
      float v[8], w[8];
      k.load(x + col, a.cols - col);
      load_weight(w, a, col, a.cols - col);
      k.get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * w[e];
      if constexpr (OUT == OUT_VALUES) {
        k.set(v);
        k.store(static_cast<T*>(a.out) + row * a.ld_out + col, a.cols - col);
      } else {
        put_codes<OUT, FMT>(a, row, col, a.cols - col, v, scale, most);
      }
    }
  }
  if constexpr (OUT == OUT_TENSOR) put_amax(a, most);
}

// ---------------------------------------------------------------------------
// COL codes: the transposed tile, each column's blocks along its rows.  Rows
// are staged in LDS as they were loaded; thread (cp, rq) then has 16 rows of the
// column pair 2 cp, and the codes go back through LDS so that they
// leave as whole 128-byte lines.  (Six waves of BF16 leave 80 VGPRs, one too few under
// delayed scaling, which spills it; five waves without the spill take the same time.)
// ---------------------------------------------------------------------------
constexpr int kColThreads = 512, kColRows = kTile / (kColThreads / 64);  // rows of a wave

template <typename T, int OUT, int FMT>
__global__ __launch_bounds__(kColThreads, sizeof(T) == 2 ? 6 : 4) void rms_columns_kernel(RmsArgs a, int tiles_x, int64_t tiles) {
  constexpr int kLoads = kTile * 16 / kColThreads;  // chunks of a thread
  __shared__ __attribute__((aligned(16))) T tile[kTile * kTile];  // rows, then codes
  __shared__ uint2 colred[kColThreads / 64][kTile / 2];
  __shared__ float rs[kTile];
  const int tid = threadIdx.x, g = tid >> 4, li = tid & 15;
  const int cp = tid & 63, rq = __builtin_amdgcn_readfirstlane(tid >> 6);
  const float scale = OUT == OUT_TENSOR ? *a.scale : 1.0f;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int64_t t = tiles - 1 - i;  // the rows written last are in the caches
    const int64_t by = t / tiles_x, row0 = by * kTile;
    const int col0 = (int)(t - by * tiles_x) * kTile;
    const int ccol = col0 + 8 * li;
    Chunk<T> k[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int64_t r = row0 + g + kColThreads / 16 * j;
      k[j].load(static_cast<const T*>(a.x) + r * a.ld_x + ccol, r < a.rows ? a.cols - ccol : 0);
    }
    const float rv = tid < kTile && row0 + tid < a.rows ? a.rstd[row0 + tid] : 0.0f;
    const int c0 = col0 + 2 * cp;
    float w0 = 1.0f, w1 = 1.0f;
    if (a.weight) {
      const int c1 = c0 + 1 < a.cols ? c0 + 1 : a.cols - 1, ca = c0 < a.cols ? c0 : a.cols - 1;
      if (a.w_bf16) {
        w0 = bf_lo(static_cast<const uint16_t*>(a.weight)[ca]);
        w1 = bf_lo(static_cast<const uint16_t*>(a.weight)[c1]);
      } else {
        w0 = static_cast<const float*>(a.weight)[ca];
        w1 = static_cast<const float*>(a.weight)[c1];
      }
    }
    if (i != blockIdx.x) __syncthreads();  // the tile before is done with
    if (tid < kTile) rs[tid] = rv;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      T* to = tile + (g + kColThreads / 16 * j) * kTile + 8 * li;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(to) = k[j].w;
      } else {
        reinterpret_cast<float4*>(to)[0] = k[j].lo;
        reinterpret_cast<float4*>(to)[1] = k[j].hi;
      }
    }
    __syncthreads();
    float u0[kColRows], u1[kColRows];
    uint32_t k0 = 0, k1 = 0;
#pragma unroll
    for (int j = 0; j < kColRows; ++j) {
      const int r = kColRows * rq + j;
      if constexpr (sizeof(T) == 2) {
        const uint32_t p = reinterpret_cast<const uint32_t*>(tile)[r * (kTile / 2) + cp];
        u0[j] = bf_lo(p);
        u1[j] = bf_hi(p);
      } else {
        const float2 p = reinterpret_cast<const float2*>(tile)[r * (kTile / 2) + cp];
        u0[j] = p.x;
        u1[j] = p.y;
      }
      u0[j] = u0[j] * rs[r] * w0;
      u1[j] = u1[j] * rs[r] * w1;
      k0 = umax32(k0, abs_key(u0[j]));
      k1 = umax32(k1, abs_key(u1[j]));
    }
    if constexpr (OUT != OUT_TENSOR) colred[rq][cp] = make_uint2(k0, k1);
    __syncthreads();  // (every wave has read the rows, too)
    if constexpr (OUT == OUT_BLOCK) {
#pragma unroll
      for (int q = 0; q < kColThreads / 64; ++q) {
        const uint2 o = colred[q][cp];
        k0 = umax32(k0, o.x);
        k1 = umax32(k1, o.y);
      }
    } else if constexpr (OUT == OUT_MX) {
      const uint2 o = colred[rq ^ 1][cp];  // the block's other 16 rows
      k0 = umax32(k0, o.x);
      k1 = umax32(k1, o.y);
    }
    const float am0 = key_to_float(k0), am1 = key_to_float(k1);
    float s0, s1;
    bool odd = false;  // a block may need the saturating encoder
    if constexpr (OUT == OUT_TENSOR) {
      s0 = s1 = scale;
      odd = !fits<FMT>(umax32(k0, k1), scale);
    } else if constexpr (OUT == OUT_BLOCK) {
      s0 = scale_from_amax<FMT>(am0, a.margin);
      s1 = scale_from_amax<FMT>(am1, a.margin);
      const bool bad0 = !is_finite(am0), bad1 = !is_finite(am1);
      odd = bad0 || bad1;
      if (rq == 0) {
        const int64_t gr = (a.rows + kTile - 1) / kTile;
        float* sc = static_cast<float*>(a.scales) + c0 * gr + by;
        if (c0 < a.cols) {
          sc[0] = recip_rn(s0);
          if (bad0 && a.nonfinite) atomicAdd(a.nonfinite, 1);
        }
        if (c0 + 1 < a.cols) {
          sc[gr] = recip_rn(s1);
          if (bad1 && a.nonfinite) atomicAdd(a.nonfinite, 1);
        }
      }
    } else {
      const int b0 = a.floor_rule ? mx_scale_byte_floor<FMT>(am0) : mx_scale_byte<FMT>(am0);
      const int b1 = a.floor_rule ? mx_scale_byte_floor<FMT>(am1) : mx_scale_byte<FMT>(am1);
      s0 = b0 == 0xFF ? 1.0f : mx_inv_scale(b0);
      s1 = b1 == 0xFF ? 1.0f : mx_inv_scale(b1);
      odd = a.floor_rule || b0 == 0xFF || b1 == 0xFF;
      if ((rq & 1) == 0 && row0 + kColRows * rq < a.rows) {
        const int64_t gr = (a.rows + 31) / 32;
        uint8_t* sc = static_cast<uint8_t*>(a.scales) + c0 * gr + 4 * by + (rq >> 1);
        if (c0 < a.cols) {
          sc[0] = (uint8_t)b0;
          if (b0 == 0xFF && a.nonfinite) atomicAdd(a.nonfinite, 1);
        }
        if (c0 + 1 < a.cols) {
          sc[gr] = (uint8_t)b1;
          if (b1 == 0xFF && a.nonfinite) atomicAdd(a.nonfinite, 1);
        }
      }
    }
    // the two columns' codes of the wave's rows
    uint32_t pk[2][kColRows / 4];
    auto encode = [&](auto Safe) __attribute__((always_inline)) {
      constexpr bool kSafe = decltype(Safe)::value;
#pragma unroll
      for (int q = 0; q < kColRows / 4; ++q) {
        pk[0][q] = encode4<FMT, kSafe>(u0[4 * q] * s0, u0[4 * q + 1] * s0, u0[4 * q + 2] * s0, u0[4 * q + 3] * s0);
        pk[1][q] = encode4<FMT, kSafe>(u1[4 * q] * s1, u1[4 * q + 1] * s1, u1[4 * q + 2] * s1, u1[4 * q + 3] * s1);
      }
    };
    // (the saturating encoder gives the same codes where it is not needed)
    if (__any(odd)) encode(std::true_type{});
    else encode(std::false_type{});
    uint8_t* ct = reinterpret_cast<uint8_t*>(tile);
#pragma unroll
    for (int half = 0; half < 2; ++half)
      *reinterpret_cast<uint4*>(ct + (2 * cp + half) * kCodeStride + kColRows * rq) =
          make_uint4(pk[half][0], pk[half][1], pk[half][2], pk[half][3]);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kTile * 8 / kColThreads; ++q) {
      const int c = (tid >> 3) + kColThreads / 8 * q, m = tid & 7;
      const int64_t left = a.rows - (row0 + 16 * m);
      if (col0 + c < a.cols && left > 0) {
        const uint4 v = *reinterpret_cast<const uint4*>(ct + c * kCodeStride + 16 * m);
        uint8_t* dst = a.q + (col0 + c) * a.ld_q + row0 + 16 * m;
        if (left >= 16) {
          __builtin_nontemporal_store(u32x4a2{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4a2*>(dst));
        } else {
          const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
          for (int j = 0; j < left; ++j) dst[j] = (uint8_t)(vw[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
template <typename T, int NT, int C, int AHEAD, bool PAST>
__global__ __launch_bounds__(threads_of(NT)) void rms_backward_kernel(RmsArgs a) {
  constexpr int kRows = threads_of(NT) / NT;
  __shared__ float red[2][16];
  int turn = 0;
  const int tid = threadIdx.x % NT;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;

  int col[C], n[C];
  float w[C][8], dw[C][8];
  Chunk<T> ct[AHEAD + 1][C], cy[AHEAD + 1][C], cd[AHEAD + 1][C];
  float rstd[AHEAD + 1];
  auto fetch = [&](int q, int64_t r) __attribute__((always_inline)) {
    if (r < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        ct[q][c].template load<PAST>(static_cast<const T*>(a.x) + r * a.ld_x + col[c], n[c]);
        cy[q][c].template load<PAST>(static_cast<const T*>(a.dy) + r * a.ld_dy + col[c], n[c]);
        if (a.residual) cd[q][c].template load<PAST>(static_cast<const T*>(a.residual) + r * a.ld_residual + col[c], n[c]);
      }
      rstd[q] = a.rstd[r];
    }
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = (c * NT + tid) * 8;
    n[c] = a.cols - col[c];
  }
#pragma unroll
  for (int q = 0; q < AHEAD; ++q) fetch(q, row + q * step);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_weight(w[c], a, col[c], n[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
  }
  for (; row < a.rows; row += step) {
    fetch(AHEAD, row + AHEAD * step);
    float s = 0.0f;  // sum of g n (dy is zero past the row's end)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float t[8], y[8];
      ct[0][c].get(t);
      cy[0][c].get(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = y[e] * (t[e] * rstd[0]);
        s += p * w[c][e];
        dw[c][e] += p;
      }
    }
    const float m = mean_of(sum_of_row<NT, sizeof(T) == 4 && NT == 512 && C == 1>(s, red, turn), a.inv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float t[8], y[8], o[8];
      ct[0][c].get(t);
      cy[0][c].get(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd[0] * (y[e] * w[c][e] - t[e] * rstd[0] * m);
      if (a.residual) {
        float d[8];
        cd[0][c].get(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += d[e];
      }
      Chunk<T> k;
      k.set(o);
      k.store(static_cast<T*>(a.out) + row * a.ld_out + col[c], n[c]);
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        ct[q][c] = ct[q + 1][c];
        cy[q][c] = cy[q + 1][c];
        cd[q][c] = cd[q + 1][c];
      }
    }
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) rstd[q] = rstd[q + 1];
  }
  if (!a.partial) return;
  float* p = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      Chunk<float> k;
      k.set(dw[c]);
      k.store(p + col[c], n[c]);
    }
  } else {
    // the workgroup's rows side by side: added here, in order
    __shared__ float sums[kRows][C * NT * 8];
    const int g = threadIdx.x / NT;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[g][col[c] + e] = dw[c][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.cols; i += threads_of(NT)) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) s += sums[r][i];
      p[i] = s;
    }
  }
}

// Rows too long for registers: dx only, two passes over each row.
template <typename T>
__global__ __launch_bounds__(1024) void rms_backward_long_kernel(RmsArgs a) {
  constexpr int NT = 1024;
  __shared__ float red[2][16];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* tr = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* yr = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const float rstd = a.rstd[row];
    float s = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
      for (int col = threadIdx.x * 8; col < a.cols; col += NT * 8) {
        Chunk<T> kt, ky;
        float t[8], y[8], w[8], o[8];
        kt.load(tr + col, a.cols - col);
        ky.load(yr + col, a.cols - col);
        load_weight(w, a, col, a.cols - col);
        kt.get(t);
        ky.get(y);
        if (pass == 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s += y[e] * (t[e] * rstd) * w[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = rstd * (y[e] * w[e] - t[e] * rstd * s);
          if (a.residual) {
            float d[8];
            kt.load(static_cast<const T*>(a.residual) + row * a.ld_residual + col, a.cols - col);
            kt.get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += d[e];
          }
          kt.set(o);
          kt.store(static_cast<T*>(a.out) + row * a.ld_out + col, a.cols - col);
        }
      }
      if (pass == 0) s = mean_of(sum_of_row<NT>(s, red, turn), a.inv);
    }
  }
}

// ... and their column sums: a wave owns 512 columns of gridDim.y-strided rows.
template <typename T>
__global__ __launch_bounds__(64) void rms_column_sums_kernel(RmsArgs a) {
  const int col = ((int)blockIdx.x * 64 + threadIdx.x) * 8, n = a.cols - col;
  if (n <= 0) return;
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    Chunk<T> kt, ky;
    float t[8], y[8];
    kt.load(static_cast<const T*>(a.x) + row * a.ld_x + col, n);
    ky.load(static_cast<const T*>(a.dy) + row * a.ld_dy + col, n);
    kt.get(t);
    ky.get(y);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] += y[e] * (t[e] * rstd);
  }
  Chunk<float> k;
  k.set(dw);
  k.store(a.partial + (int64_t)blockIdx.y * a.cols + col, n);
}

// dw from the workgroups' sums: a workgroup takes 32 columns, four to a thread,
// and each of its 128 thread groups every 128th partial.  (2^28 columns are
// 2^23 workgroups of 2^10 threads: a launch counts its work-items modulo 2^32,
// so from 2^26 columns on there are several, each with its first group.)
constexpr int kReduceCols = 32, kReduceGroups = 128;
constexpr int64_t kReduceMost = (1LL << 31) / 1024;  // workgroups of a launch
template <typename W>
__global__ __launch_bounds__(1024) void rms_reduce_kernel(const float* partial, int parts, int cols, W* dw, int64_t first) {
  __shared__ float sums[kReduceGroups][kReduceCols + 4];
  const int at = (threadIdx.x & 7) * 4, group = threadIdx.x >> 3;
  const int64_t i = (first + blockIdx.x) * kReduceCols + at, width = cols;
  float s[8] = {};
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
  if constexpr (sizeof(W) == 4) dw[j] = q;
  else dw[j] = __builtin_bit_cast(uint16_t, (__bf16)q);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Inputs that would not stay in the 256 MB Infinity Cache together are read past
// it, and so is what the forward pass leaves of them written, but for the rows
// that the launch for COL codes reads again: 8192 x 16384 with a residual 208 ->
// 194 us, into codes 278 -> 243, backward 4096 x 16384 115 -> 102.  Smaller ones
// may be there already from the kernel that made them: read past it, 4096 x 8192
// into codes 44 -> 52, 3000 x 5120 FP32 backward 49 -> 55.
bool past_caches(const RmsParams& p) {
  const int64_t inputs = 1 + (p.residual != nullptr) + (p.dy != nullptr), es = p.x_dtype == kInBf16 ? 2 : 4;
  return p.rows > (256LL << 20) / (inputs * es * p.cols);
}

RmsArgs args_of(const RmsParams& p) {
  RmsArgs a{};
  a.rows = p.rows;
  a.cols = (int)p.cols;
  a.inv = 1.0 / (double)p.cols;
  a.weight = p.weight;
  a.w_bf16 = p.w_dtype == kInBf16;
  a.eps = p.eps;
  a.rstd = p.rstd;
  a.x = p.x;
  a.ld_x = p.ld_x;
  a.residual = p.residual;
  a.ld_residual = p.ld_residual;
  a.dy = p.dy;
  a.ld_dy = p.ld_dy;
  a.total = p.total;
  a.ld_total = p.ld_total;
  a.out = p.out;
  a.ld_out = p.ld_out;
  a.margin = p.q.margin;
  a.floor_rule = p.q.recipe == kRecipeMx1x32Ocp;
  a.nonfinite = p.q.nonfinite;
  a.scale = p.q.scale;
  a.amax = reinterpret_cast<uint32_t*>(p.q.amax);
  return a;
}

template <typename T, int NT, int C, int OUT, int FMT, bool PAST, bool AGAIN>
hipError_t forward(const RmsArgs& a, hipStream_t st) {
  static std::atomic<int> occupancy{0};
  auto k = rms_forward_kernel<T, NT, C, OUT, FMT, PAST, AGAIN>;
  constexpr int threads = threads_of(NT), rows = threads / NT;
  const int64_t need = (a.rows + rows - 1) / rows;
  int64_t most = resident(k, threads, occupancy, st);
  if (OUT == OUT_TENSOR && most > kAmaxSlots) most = kAmaxSlots;
  k<<<(unsigned)(need < most ? need : most), threads, 0, st>>>(a);
  return hipGetLastError();
}

// Threads of a row, chunks of 8 columns of a thread.  Short rows by 16 lanes, four
// of them in a wave: 262144 x 128 BF16 60 -> 23 us against a wave per row, into
// codes 77 -> 22, backward 120 -> 41; 131072 x 256 33 -> 23, 41 -> 21, 73 -> 40.
template <typename T, int OUT, int FMT, bool PAST, bool AGAIN>
hipError_t forward_cols(const RmsArgs& a, hipStream_t st) {
  if (a.cols <= 128) return forward<T, 16, 1, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= kShort) return forward<T, 16, 2, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= 512) return forward<T, 64, 1, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= kMiddle) return forward<T, 64, 2, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= 2048) return forward<T, 256, 1, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= 4096) return forward<T, 256, 2, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= 8192) return forward<T, 512, 2, OUT, FMT, PAST, AGAIN>(a, st);
  if (a.cols <= 16384) return forward<T, 1024, 2, OUT, FMT, PAST, AGAIN>(a, st);
  int64_t most = 2 * (int64_t)cu_count(stream_device(st));
  if (OUT == OUT_TENSOR && most > kAmaxSlots) most = kAmaxSlots;
  rms_forward_long_kernel<T, OUT, FMT><<<(unsigned)(a.rows < most ? a.rows : most), 1024, 0, st>>>(a);
  return hipGetLastError();
}

// (codes alone and values are not read again: with those of both orientations t is)
template <typename T, int OUT, int FMT, bool AGAIN>
hipError_t forward_any(const RmsArgs& a, bool past, hipStream_t st) {
  return past ? forward_cols<T, OUT, FMT, true, AGAIN>(a, st) : forward_cols<T, OUT, FMT, false, AGAIN>(a, st);
}

template <typename T, int OUT, int FMT>
hipError_t columns(const RmsArgs& a, hipStream_t st) {
  static std::atomic<int> occupancy{0};
  auto k = rms_columns_kernel<T, OUT, FMT>;
  const int64_t tiles_x = (a.cols + kTile - 1) / kTile, tiles = tiles_x * ((a.rows + kTile - 1) / kTile);
  const int64_t most = resident(k, kColThreads, occupancy, st), rounds = (tiles + most - 1) / most;
  k<<<(unsigned)((tiles + rounds - 1) / rounds), kColThreads, 0, st>>>(a, (int)tiles_x, tiles);
  return hipGetLastError();
}

template <typename T, int OUT, int FMT>
hipError_t quantize(const RmsParams& p, hipStream_t st) {
  RmsArgs a = args_of(p);
  a.q = p.q.orient & 1 ? p.q.q_row : nullptr;
  a.ld_q = p.q.ld_q_row;
  a.scales = p.q.s_row;
  const bool past = past_caches(p), col = p.q.orient & 2;
  if (!col) return forward_any<T, OUT, FMT, false>(a, past, st);
  // (delayed scaling takes the maximum of y whatever the orientation)
  const hipError_t e = p.q.orient & 1 || OUT == OUT_TENSOR ? forward_any<T, OUT, FMT, true>(a, past, st)
                                                           : forward_any<T, OUT_VALUES, kE4M3, true>(a, past, st);
  if (e != hipSuccess) return e;
  if (p.residual) {
    a.x = p.total;
    a.ld_x = p.ld_total;
  }
  a.q = p.q.q_col;
  a.ld_q = p.q.ld_q_col;
  a.scales = p.q.s_col;
  return columns<T, OUT, FMT>(a, st);
}

template <typename T>
hipError_t quantize_any(const RmsParams& p, hipStream_t st) {
  const bool block = p.q.recipe == kRecipeBlock1x128;
  if (p.q.recipe == kRecipeTensorDelayed)
    return p.q.fmt == kE4M3 ? quantize<T, OUT_TENSOR, kE4M3>(p, st) : quantize<T, OUT_TENSOR, kE5M2>(p, st);
  if (p.q.fmt == kE4M3) return block ? quantize<T, OUT_BLOCK, kE4M3>(p, st) : quantize<T, OUT_MX, kE4M3>(p, st);
  return block ? quantize<T, OUT_BLOCK, kE5M2>(p, st) : quantize<T, OUT_MX, kE5M2>(p, st);
}

template <typename W>
hipError_t reduce(const RmsParams& p, int parts, hipStream_t st) {
  if (!p.dweight) return hipGetLastError();
  const int64_t groups = (p.cols + kReduceCols - 1) / kReduceCols;
  for (int64_t g = 0; g < groups; g += kReduceMost) {
    const int64_t n = groups - g < kReduceMost ? groups - g : kReduceMost;
    rms_reduce_kernel<W><<<(unsigned)n, 1024, 0, st>>>(p.workspace, parts, (int)p.cols, static_cast<W*>(p.dweight), g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t reduce_any(const RmsParams& p, int parts, hipStream_t st) {
  return p.w_dtype == kInBf16 ? reduce<uint16_t>(p, parts, st) : reduce<float>(p, parts, st);
}

template <typename T, int NT, int C, int AHEAD, bool PAST>
hipError_t backward(const RmsParams& p, hipStream_t st) {
  static std::atomic<int> occupancy{0};
  auto k = rms_backward_kernel<T, NT, C, AHEAD, PAST>;
  constexpr int threads = threads_of(NT);
  int64_t blocks = rms_partials(p.rows, p.cols);
  const int64_t most = resident(k, threads, occupancy, st);
  blocks = blocks < most ? blocks : most;
  RmsArgs a = args_of(p);
  a.partial = p.dweight ? p.workspace : nullptr;
  k<<<(unsigned)blocks, threads, 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : reduce_any(p, (int)blocks, st);
}

template <typename T, bool PAST>
hipError_t backward_cols(const RmsParams& p, hipStream_t st) {
  if (p.cols <= 128) return backward<T, 16, 1, 1, PAST>(p, st);
  if (p.cols <= kShort) return backward<T, 16, 2, 1, PAST>(p, st);
  if (p.cols <= 512) return backward<T, 64, 1, 1, PAST>(p, st);
  if (p.cols <= kMiddle) return backward<T, 64, 2, 1, PAST>(p, st);
  if (p.cols <= 2048) return backward<T, 256, 1, 2, PAST>(p, st);
  // (FP32, 256 threads of two chunks or 512 of one: 1000 x 4000 16.5 and 15.3 us, 2000
  // x 4000 29.3 and 27.4, 8192 x 4096 84 and 83; BF16 8192 x 4096 52.1 and 54.0)
  if (p.cols <= 4096) return backward<T, sizeof(T) == 4 ? 512 : 256, sizeof(T) == 4 ? 1 : 2, 2, PAST>(p, st);
  if (p.cols <= 8192) return backward<T, 512, 2, 2, PAST>(p, st);
  return backward<T, 1024, 2, 0, PAST>(p, st);
}

template <typename T>
hipError_t backward_any(const RmsParams& p, hipStream_t st) {
  if (p.rows == 0) return reduce_any(p, 0, st);
  if (p.cols <= 16384) return past_caches(p) ? backward_cols<T, true>(p, st) : backward_cols<T, false>(p, st);
  const int64_t most = 2 * (int64_t)cu_count(stream_device(st));
  RmsArgs a = args_of(p);
  rms_backward_long_kernel<T><<<(unsigned)(p.rows < most ? p.rows : most), 1024, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.dweight) return e;
  a.partial = p.workspace;
  const int64_t parts = rms_partials(p.rows, p.cols);
  rms_column_sums_kernel<T><<<dim3((unsigned)((p.cols + 511) / 512), (unsigned)parts), 64, 0, st>>>(a);
  e = hipGetLastError();
  return e != hipSuccess ? e : reduce_any(p, (int)parts, st);
}

}  // namespace

// sets of column sums that a backward pass over `rows` rows may leave
int64_t rms_partials(int64_t rows, int64_t cols) {
  const int64_t per = rows_per_partial(rows, cols), n = rows / per + (rows % per != 0);
  const int64_t most = cols <= kShort ? kMaxShortPartials : kMaxPartials;
  return n < 1 ? 1 : (n < most ? n : most);
}

hipError_t launch_rms_forward(const RmsParams& p, hipStream_t st) {
  const RmsArgs a = args_of(p);
  const bool past = past_caches(p);
  return p.x_dtype == kInBf16 ? forward_any<uint16_t, OUT_VALUES, kE4M3, false>(a, past, st)
                              : forward_any<float, OUT_VALUES, kE4M3, false>(a, past, st);
}

hipError_t launch_rms_quantize(const RmsParams& p, hipStream_t st) {
  return p.x_dtype == kInBf16 ? quantize_any<uint16_t>(p, st) : quantize_any<float>(p, st);
}

hipError_t launch_rms_backward(const RmsParams& p, hipStream_t st) {
  return p.x_dtype == kInBf16 ? backward_any<uint16_t>(p, st) : backward_any<float>(p, st);
}

}  // namespace fp8mi
