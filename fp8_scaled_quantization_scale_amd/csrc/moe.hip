// moe.hip -- tokens sorted by expert and back, for gfx950: the sort, the plain
// dispatch, the weighted combine and its gradient.  (The dispatch into FP8
// codes reads through the sort's row map in quantize.hip: moe_tile_kernel for
// BF16 rows of whole tiles, the MOE form of quant_tile_kernel for the others.)
//
// Slot s = t topk + j is token t's j-th choice.  The sorted buffer holds one
// segment per expert, each starting on a multiple of 128 rows, so that a
// 128-row block of column scales, a K window of the weight gradient and a row
// tile never hold two experts' rows; the rows after a segment's last slot are
// zero.  Slots whose expert is outside [0, experts) have no row.
#include "launch.hpp"
#include "rows.hpp"

namespace fp8mi {

namespace {

// ---------------------------------------------------------------------------
// Sort: a stable counting sort.  A workgroup takes a range of slots, a wave a
// part of it.  With more than one workgroup a first launch counts each range's
// slots per expert; in the second each workgroup adds up the counts of all
// ranges (the segments' sizes) and of those before its own, turns its waves'
// counts into first rows, and every wave then walks its part in order, 64
// slots at a time: equal experts among the 64 lanes find each other with one
// ballot per bit of the number.  No atomic decides an order: those on LDS
// only count.  Bound by latency: 256 slots over 8 experts 4.1 us (one launch),
// 65536 over 64 in 4.9 + 6.2 us (13.5 for the second with the ranges' counts
// added up by one thread per expert and the experts read twice).
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortRange = 2048;   // slots per workgroup, until there would be
constexpr int kSortMaxBlocks = 256;  // more workgroups than this

struct SortArgs {
  const void* expert;
  int64_t ld;
  int topk, experts, blocks;
  int64_t slots, range, rows;
  int32_t *offsets, *counts, *row_slot, *slot_row;
  int32_t* hist;  // [blocks][experts], with more than one workgroup
};

// expert of slot s, -1 if it has none
template <typename Idx>
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t s) {
  const Idx* p = static_cast<const Idx*>(a.expert);
  Idx v;
  if (a.ld == a.topk) {
    v = p[s];
  } else {
    const uint32_t t = (uint32_t)s / (uint32_t)a.topk;
    v = p[(int64_t)t * a.ld + ((uint32_t)s - t * (uint32_t)a.topk)];
  }
  return v >= 0 && v < a.experts ? (int)v : -1;
}

template <typename Idx>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int cnt[kMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * a.range, to = min(from + a.range, a.slots);
  for (int64_t s = from + threadIdx.x; s < to; s += kSortThreads) {
    const int e = expert_of<Idx>(a, s);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.hist[(int64_t)blockIdx.x * a.experts + e] = cnt[e];
}

// PER: slots per lane, whose experts stay in registers from the count to the
// walk (0: any number, read twice).
template <typename Idx, int PER>
__global__ __launch_bounds__(kSortThreads) void sort_rows_kernel(SortArgs a) {
  extern __shared__ int cnt[];  // [kSortWaves][experts]: counts, then the next row of each
  __shared__ int sums[2][kSortThreads];  // parts of the ranges' sums
  __shared__ int at[kMaxExperts + 1];  // segment starts
  __shared__ int total[kMaxExperts];
  __shared__ int wave_total[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t part = a.range / kSortWaves;  // a multiple of 64
  const int64_t from = blockIdx.x * a.range + wave * part, to = min(from + part, a.slots);

  for (int i = tid; i < kSortWaves * a.experts; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int held[PER ? PER : 1];
  if constexpr (PER > 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) held[i] = from + 64 * i + lane < to ? expert_of<Idx>(a, from + 64 * i + lane) : -1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (held[i] >= 0) atomicAdd(&cnt[wave * a.experts + held[i]], 1);
  } else {
    for (int64_t s = from + lane; s < to; s += 64) {
      const int e = expert_of<Idx>(a, s);
      if (e >= 0) atomicAdd(&cnt[wave * a.experts + e], 1);
    }
  }
  // the ranges' counts, added up by as many threads per expert as there are
  const int wide = a.experts > 1 ? 1 << (32 - __clz(a.experts - 1)) : 1;  // experts, up to a power of two
  const int groups = min(kSortThreads / wide, 32);
  if (a.blocks > 1) {
    const int x = tid & (wide - 1), part = tid / wide;
    int all = 0, before = 0;
    if (x < a.experts && part < groups)
      for (int b = part; b < a.blocks; b += groups) {
        const int n = a.hist[(int64_t)b * a.experts + x];
        all += n;
        before += b < (int)blockIdx.x ? n : 0;
      }
    sums[0][tid] = all;
    sums[1][tid] = before;
  }
  __syncthreads();

  // segment sizes, and the rows of a segment that earlier workgroups fill
  const int e = tid;
  int mine = 0, before = 0, all = 0;
  if (e < a.experts) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) mine += cnt[w * a.experts + e];
    if (a.blocks == 1) {
      all = mine;
    } else {
      for (int g = 0; g < groups; ++g) {
        all += sums[0][g * wide + e];
        before += sums[1][g * wide + e];
      }
    }
  }
  // scan of the padded sizes over the experts, one per thread
  const int padded = (all + kExpertAlign - 1) / kExpertAlign * kExpertAlign;
  int scan = padded;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(scan, off, 64);
    if (lane >= off) scan += o;
  }
  if (lane == 63) wave_total[wave] = scan;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < wave; ++w) base += wave_total[w];
  const int start = base + scan - padded;
  if (e < a.experts) {
    at[e + 1] = start + padded;
    total[e] = all;
    int row = start + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = cnt[w * a.experts + e];
      cnt[w * a.experts + e] = row;
      row += n;
    }
    if (blockIdx.x == 0) {
      a.offsets[e + 1] = start + padded;
      a.counts[e] = all;
    }
  }
  if (tid == 0) {
    at[0] = 0;
    if (blockIdx.x == 0) a.offsets[0] = 0;
  }
  __syncthreads();

  // rows of this wave's slots, in order
  const int bits = 32 - __clz(a.experts);  // of an expert's number plus one
  volatile int* next = cnt + wave * a.experts;
  auto walk = [&](int64_t s, int k) __attribute__((always_inline)) {
    uint64_t same = ~0ull;  // lanes with this lane's expert
    for (int b = 0; b < bits; ++b) {
      const bool set = ((k + 1) >> b) & 1;
      const uint64_t m = __ballot(set);
      same &= set ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (k >= 0) row = next[k] + rank;
    __builtin_amdgcn_wave_barrier();
    if (k >= 0 && rank == 0) next[k] = row + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (s < to) {
      a.slot_row[s] = row;
      if (row >= 0 && row < a.rows) a.row_slot[row] = (int)s;
    }
  };
  if constexpr (PER > 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) walk(from + 64 * i + lane, held[i]);
  } else {
    for (int64_t s0 = from; s0 < to; s0 += 64) walk(s0 + lane, s0 + lane < to ? expert_of<Idx>(a, s0 + lane) : -1);
  }

  // rows that hold no slot: the segments' ends, and what lies behind the last
  for (int x = blockIdx.x * kSortWaves + wave; x < a.experts; x += a.blocks * kSortWaves) {
    for (int r = at[x] + total[x] + lane; r < at[x + 1]; r += 64)
      if (r < a.rows) a.row_slot[r] = -1;
  }
  for (int64_t r = at[a.experts] + (int64_t)blockIdx.x * kSortThreads + tid; r < a.rows; r += (int64_t)a.blocks * kSortThreads)
    a.row_slot[r] = -1;
}

// ---------------------------------------------------------------------------
// Rows to and from the sorted buffer.  All three are bound by memory (16384 x
// 8192 to 4 experts each: dispatch 286 us, 4.9 TB/s; combine 237 us, 5.7 TB/s;
// the gradient of 4095 x 4096 to 8: 117 us, 4.8 TB/s and 33 MB of pads); a wave
// works on one token's (or one pad row's) piece of 64 chunks x kPiece, so the
// token's row numbers and weights are the same for all its lanes.
//
// Outputs of dispatch and combine that would fill half the 256 MB Infinity
// Cache by themselves are written past it (combine 16384 x 8192 of 4: 256 -> 237
// us; 8192 x 4096 of 2, whose output a next kernel finds there: 36.0 us, past it
// 38.1), the gradient's sorted rows always are (4095 x 4096 of 8: 125 -> 118 us,
// 300 x 1024 of 8: 10.1 -> 8.6).  512 threads: the gradient of 4095 x 4096 took
// 131 us with 256 and 148 with 128, the others the same.
// ---------------------------------------------------------------------------
constexpr int kPiece = 2;                       // chunks of 8 elements per lane
constexpr int kPieceCols = 64 * 8 * kPiece;     // columns of a piece
constexpr int kRowThreads = 512, kRowWaves = kRowThreads / 64;

struct RowArgs {
  int64_t tokens, cols, rows, ld_token, ld_expert, ld_out;
  int topk, experts, pieces;  // pieces of a row
  const int32_t *offsets, *counts, *slot_row;
  const float* weights;
  const void* token_rows;
  const void* expert_rows;
  void* out;
  float* dweights;
  int64_t first;  // piece (combine's gradient: token) that the launch starts at
};

// Zeros in the rows of the sorted buffer that hold no slot, expert x's.
template <typename T>
__device__ __forceinline__ void zero_pads(const RowArgs& a, int x) {
  const int64_t from = (int64_t)a.offsets[x] + a.counts[x], to = min((int64_t)a.offsets[x + 1], a.rows);
  Chunk<T> z;
  z.fill(0.0f);
  for (int64_t r = max(from, (int64_t)0) + (threadIdx.x >> 6); r < to; r += kRowWaves)
    for (int64_t c = (threadIdx.x & 63) * 8; c < a.cols; c += 64 * 8)
      z.store(static_cast<T*>(a.out) + r * a.ld_out + c, a.cols - c);
}

// out[row(t, j)] = w_tj x[t]
template <typename T, bool NT>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(RowArgs a, int64_t token_blocks) {
  if ((int64_t)blockIdx.x >= token_blocks) return zero_pads<T>(a, (int)(blockIdx.x - token_blocks));
  const int lane = threadIdx.x & 63;
  const int64_t unit = a.first + (int64_t)blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = unit / a.pieces;
  if (t >= a.tokens) return;
  const int64_t c0 = (unit - t * a.pieces) * kPieceCols + lane * 8;
  Chunk<T> k[kPiece];
#pragma unroll
  for (int i = 0; i < kPiece; ++i)
    k[i].load(static_cast<const T*>(a.token_rows) + t * a.ld_token + c0 + i * 512, a.cols - (c0 + i * 512));
  for (int j = 0; j < a.topk; ++j) {
    const int64_t row = a.slot_row[t * a.topk + j];
    if (row < 0 || row >= a.rows) continue;
    T* dst = static_cast<T*>(a.out) + row * a.ld_out;
    const float w = a.weights ? a.weights[t * a.topk + j] : 1.0f;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
      Chunk<T> o = k[i];
      if (a.weights) {
        float v[8];
        o.get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w;
        o.set(v);
      }
      o.template store<NT>(dst + c0 + i * 512, a.cols - (c0 + i * 512));
    }
  }
}

// y[t] = sum_j w_tj ys[row(t, j)], in FP32
template <typename T, bool NT>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = a.first + (int64_t)blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = unit / a.pieces;
  if (t >= a.tokens) return;
  const int64_t c0 = (unit - t * a.pieces) * kPieceCols + lane * 8;
  float acc[kPiece][8];
#pragma unroll
  for (int i = 0; i < kPiece; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
  constexpr int kAtOnce = 4;  // rows on their way together
  for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
    Chunk<T> k[kAtOnce][kPiece];
    float w[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      const int64_t slot = t * a.topk + j0 + q;
      const int64_t row = j0 + q < a.topk ? a.slot_row[slot] : -1;
      const bool there = row >= 0 && row < a.rows;
      w[q] = there ? (a.weights ? a.weights[slot] : 1.0f) : 0.0f;
      // (a slot without a row adds 0 * 0)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        k[q][i].fill(0.0f);
        if (there)
          k[q][i].load(static_cast<const T*>(a.expert_rows) + row * a.ld_expert + c0 + i * 512, a.cols - (c0 + i * 512));
      }
    }
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) {
        float v[8];
        k[q][i].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] += w[q] * v[e];
      }
  }
#pragma unroll
  for (int i = 0; i < kPiece; ++i) {
    Chunk<T> o;
    o.set(acc[i]);
    o.template store<NT>(static_cast<T*>(a.out) + t * a.ld_out + c0 + i * 512, a.cols - (c0 + i * 512));
  }
}

// out[row(t, j)] = w_tj dy[t] (if out), dweights_tj = <dy[t], ys[row(t, j)]>
// (if dweights): NT threads per token, so that each dot product ends inside a
// wave (NT 64) or a workgroup.  Up to kWaveCols columns a wave: a workgroup would
// be mostly idle (8192 tokens, 512 columns to 2: 13 us against 77; 1024 to 8: 60
// against 109; 2048 to 4: 74 against 100; but 4095 x 4096 to 8: 139 against 120).
constexpr int kWaveCols = 2048;
template <typename T, int NT>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(RowArgs a, int64_t token_blocks) {
  if ((int64_t)blockIdx.x >= token_blocks) return zero_pads<T>(a, (int)(blockIdx.x - token_blocks));
  constexpr int kAtOnce = 8;
  __shared__ float red[kRowWaves][kAtOnce];
  const int tid = threadIdx.x % NT;
  const int64_t t = a.first + (int64_t)blockIdx.x * (kRowThreads / NT) + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  if (t >= a.tokens) return;  // (whole waves; a workgroup of one token has it)
  const T* dy = static_cast<const T*>(a.token_rows) + t * a.ld_token;
  for (int j0 = 0; j0 < a.topk; j0 += kAtOnce) {
    float dot[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) dot[q] = 0.0f;
    // the group's rows and weights, the same for the whole workgroup
    int64_t row[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      const int64_t slot = t * a.topk + j0 + q;
      row[q] = j0 + q < a.topk ? a.slot_row[slot] : -1;
      if (row[q] >= a.rows) row[q] = -1;
      w[q] = a.weights && j0 + q < a.topk ? a.weights[slot] : 1.0f;
    }
    for (int64_t c = tid * 8; c < a.cols; c += NT * 8) {
      Chunk<T> k, y[kAtOnce];  // all on their way together
      float g[8];
      k.load(dy + c, a.cols - c);
      if (a.dweights) {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          y[q].fill(0.0f);
          if (row[q] >= 0) y[q].load(static_cast<const T*>(a.expert_rows) + row[q] * a.ld_expert + c, a.cols - c);
        }
      }
      k.get(g);
      if (a.out) {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          if (row[q] < 0) continue;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = g[e] * w[q];
          k.set(v);
          k.template store<true>(static_cast<T*>(a.out) + row[q] * a.ld_out + c, a.cols - c);
        }
      }
      if (a.dweights) {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          float v[8];
          y[q].get(v);
          if (row[q] >= 0) {  // (a non-finite dy times no row is nothing)
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[q] += g[e] * v[e];
          }
        }
      }
    }
    if (!a.dweights) continue;
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) dot[q] = wave_sum(dot[q]);
    if constexpr (NT == 64) {
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (tid == 0 && j0 + q < a.topk) a.dweights[t * a.topk + j0 + q] = dot[q];
    } else {
      __syncthreads();  // red is read below before the next group's sums
      if ((tid & 63) == 0) {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) red[tid >> 6][q] = dot[q];
      }
      __syncthreads();
      const int q = tid;
      if (q < kAtOnce && j0 + q < a.topk) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) s += red[w][q];
        a.dweights[t * a.topk + j0 + q] = s;  // 0 for a slot without a row
      }
    }
  }
}

RowArgs args_of(const MoeRowsParams& p) {
  return RowArgs{p.tokens,       p.cols,       p.rows,
                 p.ld_token,     p.ld_expert,  p.ld_out,
                 (int)p.topk,    (int)p.experts, (int)((p.cols + kPieceCols - 1) / kPieceCols),
                 p.offsets,      p.counts,     p.slot_row,
                 p.weights,      p.token_rows, p.expert_rows,
                 p.out,          p.dweights,   0};
}

// A launch has its work-items counted modulo 2^32: `groups` workgroups of
// kRowThreads go out as launches of at most this many, each with the first of
// its pieces (or tokens), `per` to a workgroup.  launch(args, groups, whether
// it is the first launch).
constexpr int64_t kMostGroups = (1LL << 31) / kRowThreads;
template <typename Launch>
hipError_t in_parts(RowArgs a, int64_t groups, int per, Launch&& launch) {
  for (int64_t g = 0; g < groups; g += kMostGroups) {
    a.first = g * per;
    launch(a, groups - g < kMostGroups ? groups - g : kMostGroups, g == 0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// whether `rows` rows of output are written past the caches
bool past_caches(int64_t rows, const MoeRowsParams& p) {
  return rows * p.cols * (p.dtype == kInBf16 ? 2 : 4) > (128LL << 20);
}

int64_t sort_range(int64_t slots) {
  const int64_t least = (slots + kSortMaxBlocks - 1) / kSortMaxBlocks;
  const int64_t range = least > kSortRange ? least : kSortRange;
  return (range + kSortThreads - 1) / kSortThreads * kSortThreads;
}

template <typename Idx>
hipError_t sort_any(const MoeSortParams& p, hipStream_t st) {
  SortArgs a;
  a.expert = p.expert;
  a.ld = p.ld_expert;
  a.topk = (int)p.topk;
  a.experts = (int)p.experts;
  a.slots = p.tokens * p.topk;
  a.range = sort_range(a.slots);
  a.blocks = (int)moe_sort_blocks(a.slots);
  a.rows = p.rows;
  a.offsets = p.offsets;
  a.counts = p.counts;
  a.row_slot = p.row_slot;
  a.slot_row = p.slot_row;
  a.hist = p.workspace;
  if (a.blocks > 1) {
    sort_count_kernel<Idx><<<(unsigned)a.blocks, kSortThreads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t lds = kSortWaves * a.experts * sizeof(int);
  if (a.range == kSortRange) sort_rows_kernel<Idx, kSortRange / kSortThreads><<<(unsigned)a.blocks, kSortThreads, lds, st>>>(a);
  else sort_rows_kernel<Idx, 0><<<(unsigned)a.blocks, kSortThreads, lds, st>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t moe_sort_blocks(int64_t slots) {
  const int64_t n = (slots + sort_range(slots) - 1) / sort_range(slots);
  return n < 1 ? 1 : n;
}

hipError_t launch_moe_sort(const MoeSortParams& p, hipStream_t st) {
  return p.idx_dtype == 0 ? sort_any<int32_t>(p, st) : sort_any<int64_t>(p, st);
}

hipError_t launch_moe_dispatch(const MoeRowsParams& p, hipStream_t st) {
  const RowArgs all = args_of(p);
  const bool past = past_caches(p.tokens * p.topk, p);
  return in_parts(all, (p.tokens * all.pieces + kRowWaves - 1) / kRowWaves, kRowWaves,
                  [&](const RowArgs& a, int64_t blocks, bool pads) {
    const unsigned grid = (unsigned)(blocks + (pads ? p.experts : 0));
    if (p.dtype == kInBf16)
      past ? dispatch_kernel<uint16_t, true><<<grid, kRowThreads, 0, st>>>(a, blocks)
           : dispatch_kernel<uint16_t, false><<<grid, kRowThreads, 0, st>>>(a, blocks);
    else
      past ? dispatch_kernel<float, true><<<grid, kRowThreads, 0, st>>>(a, blocks)
           : dispatch_kernel<float, false><<<grid, kRowThreads, 0, st>>>(a, blocks);
  });
}

hipError_t launch_moe_combine(const MoeRowsParams& p, hipStream_t st) {
  const RowArgs all = args_of(p);
  const bool past = past_caches(p.tokens, p);
  return in_parts(all, (p.tokens * all.pieces + kRowWaves - 1) / kRowWaves, kRowWaves,
                  [&](const RowArgs& a, int64_t blocks, bool) {
    const unsigned grid = (unsigned)blocks;
    if (p.dtype == kInBf16)
      past ? combine_kernel<uint16_t, true><<<grid, kRowThreads, 0, st>>>(a)
           : combine_kernel<uint16_t, false><<<grid, kRowThreads, 0, st>>>(a);
    else
      past ? combine_kernel<float, true><<<grid, kRowThreads, 0, st>>>(a)
           : combine_kernel<float, false><<<grid, kRowThreads, 0, st>>>(a);
  });
}

hipError_t launch_moe_combine_backward(const MoeRowsParams& p, hipStream_t st) {
  const bool wave = p.cols <= kWaveCols;
  const int per = wave ? kRowWaves : 1;
  return in_parts(args_of(p), (p.tokens + per - 1) / per, per, [&](const RowArgs& a, int64_t blocks, bool pads) {
    const unsigned grid = (unsigned)(blocks + (pads && p.out ? p.experts : 0));
    if (p.dtype == kInBf16)
      wave ? combine_backward_kernel<uint16_t, 64><<<grid, kRowThreads, 0, st>>>(a, blocks)
           : combine_backward_kernel<uint16_t, kRowThreads><<<grid, kRowThreads, 0, st>>>(a, blocks);
    else
      wave ? combine_backward_kernel<float, 64><<<grid, kRowThreads, 0, st>>>(a, blocks)
           : combine_backward_kernel<float, kRowThreads><<<grid, kRowThreads, 0, st>>>(a, blocks);
  });
}

}  // namespace fp8mi
