// route.hip -- the experts' router for gfx950: softmax over the experts, the
// choice of the topk largest, their weights, the slots of each expert and the
// balance loss, with the logits' gradient.
//
//   p = softmax(l), loss = experts sum_e f_e P_e,
//   f_e = counts_e / (n topk), P_e = sum over tokens of p_te / n, n tokens,
//   slope_e = d loss / d p_te = experts f_e / n (the counts have no gradient),
//   dp = dloss slope + (the weights' part), dl = p (dp - <p, dp>).
//
// G lanes own a token (16 up to 256 experts, so that a maximum or a sum over them
// is one of V registers and four DPP rotations; above, a wave), V experts each, in
// vectors of at most 16 bytes of which the lanes' lie side by side.  The next
// token's logits are on their way while one is worked on.
//
// The choice.  Logits are compared as integers that order like them, with the
// expert's number in the low bits so that no two are equal (of equal logits the
// lowest expert is the largest).  The next choice is then the largest integer
// below the last one: the largest difference to it modulo 2^32, one subtraction
// and half a three-way maximum per expert, and nothing is marked as taken.  FP32
// logits lose as many low bits as an expert's number has: where two of a token's
// topk + 1 largest are equal without them, and where a NaN, an infinity or the
// lowest values are among the chosen, the wave chooses once more by whole
// integers (choose_exact), as it does for more than 16 choices.
//
// Sums over the tokens are taken in registers, then over the workgroup and, by a
// second launch in a fixed order, over all workgroups; only integers are counted
// with atomics.
//
// Measured (MI355X): forward 65536 x 256 BF16 to 8 26 + 5 us, bound by
// instructions (718 per four tokens, 300 of them the choice, 19 us of issue; the
// logits' 34 MB would take 6 us; choosing by marking what is taken cost 26 us more);
// 16384 x 64 FP32 to 4 6 + 4.5 us and 128 x 8 to 2 4.4 us (one launch), latency.
// Gradient 65536 x 256 FP32 31 us (4.3 TB/s), 16384 x 64 5.6 us.
#include "launch.hpp"
#include "rows.hpp"
#include "tile.hpp"

namespace fp8mi {

namespace {

constexpr int kRouteMaxBlocks = 256;
// Tokens per group of lanes up to which there is one workgroup, and one launch
// (128 x 8 4.7 us; of 64 tokens each, with the second launch, 6.2).
constexpr int kRouteOneBlock = 4;

// lanes that own a token, and the experts of a lane: the power of two that they
// hold them with
constexpr int lanes_of(int64_t experts) { return experts <= 256 ? 16 : 64; }
constexpr int per_lane(int64_t experts) {
  int v = 1;
  while (lanes_of(experts) * v < experts) v *= 2;
  return v;
}
constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }
constexpr int kRouteThreads = 1024;

struct RouteArgs {
  const void* logits;
  int64_t tokens, ld;
  int experts, topk, normalize, blocks;
  const uint8_t* mask;
  int32_t* expert;
  float* weights;
  const void* chosen;
  int wide;  // chosen is int64
  int64_t ld_chosen;
  float* loss;
  int32_t* counts;
  float* slope;
  // the workgroups' sums
  float* psum;        // [blocks][experts]
  int32_t* hist;      // [blocks][experts]
  int32_t* held;      // [blocks] tokens
  float* part;        // [32] of the loss
  uint32_t* ticket;
  const float* dweights;
  const float* dloss;
  void* dlogits;
  int64_t ld_dlogits;
};

__device__ __forceinline__ float as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t as_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

// over the G lanes of a token; all of them get it
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
  v += as_float(dpp<0x128>(as_bits(v)));
  v += as_float(dpp<0x124>(as_bits(v)));
  v += as_float(dpp<0x122>(as_bits(v)));
  v += as_float(dpp<0x121>(as_bits(v)));
  if constexpr (G == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}
template <int G>
__device__ __forceinline__ float lanes_fmax(float v) {
  v = fmaxf(v, as_float(dpp<0x128>(as_bits(v))));
  v = fmaxf(v, as_float(dpp<0x124>(as_bits(v))));
  v = fmaxf(v, as_float(dpp<0x122>(as_bits(v))));
  v = fmaxf(v, as_float(dpp<0x121>(as_bits(v))));
  if constexpr (G == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = row16_max(v);
  if constexpr (G == 64) {  // (the four rows' are scalars)
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    v = umax32(umax32(a, b), umax32(c, d));
  }
  return v;
}

constexpr float kNegInf = -__builtin_inff();

// an integer that orders like the logit, NaN on top; 0: not to be chosen (-inf)
__device__ __forceinline__ uint32_t key_of(float v) {
  v += 0.0f;  // -0 is 0
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = as_bits(v);
  return __builtin_elementwise_sub_sat(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 0x007FFFFFu);
}

// e^d with d = v - most, at most 0: d log2(e) = n + r with n whole, at least -126,
// and 2^r 2^n.  r is rounded as the small number that it is (log2(e) in two parts,
// the second as an fma), so that the result is off by 2.4 half steps, and what v -
// most loses, at any distance (2^(d log2(e)) with the product rounded to FP32 takes a
// third of the instructions and 65536 x 256 from 28.5 to 26 us, but is off by 32 half
// steps at 20 to 40 below the largest, which a weight, a gradient and the loss of
// choices that lie there show).  Below 2^-126 r takes the rest, and the product is
// denormal; -inf is 0.
__device__ __forceinline__ float weight_of(float v, float most) {
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kWhole = 0x1.8p+23f;
  const float d = v - most;
  const float t = __builtin_fmaf(fmaxf(d, -87.0f), kLog2e, kWhole);  // (its low bits are n)
  const float n = t - kWhole;
  const float r = __builtin_fmaf(d, kRest, __builtin_fmaf(d, kLog2e, -n));
  return __builtin_amdgcn_exp2f(r) * as_float((as_bits(t) << 23) + 0x3F800000u);
}

// A lane's experts: vectors of kWide, G lanes of them and then the next.  expert()
// is the number of the i-th without the lane's part, which is lane() and shares
// no bit with it.
template <typename T, int G, int V>
struct Own {
  static constexpr int kWide = V < 16 / (int)sizeof(T) ? V : 16 / (int)sizeof(T);
  typedef T vec __attribute__((ext_vector_type(kWide < 2 ? 2 : kWide), aligned(sizeof(T))));
  static constexpr __host__ __device__ int expert(int i) { return i / kWide * G * kWide + i % kWide; }
  static __device__ __forceinline__ int lane() { return (threadIdx.x & (G - 1)) * kWide; }
};

// V logits as they lie in memory, of which those below n - lane() are there.
// EVEN: the number of experts is a multiple of kWide, so that no vector is cut.
template <typename T, int G, int V, bool EVEN>
struct Logits {
  using O = Own<T, G, V>;
  typename O::vec c[V / O::kWide];
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int k = 0; k < V / O::kWide; ++k) {
      const T* q = p + O::expert(k * O::kWide);
      const int left = n - O::expert(k * O::kWide);
      if constexpr (O::kWide == 1) {
        if (left > 0) c[k][0] = *q;
      } else if (EVEN ? left > 0 : left >= O::kWide) {
        c[k] = *reinterpret_cast<const typename O::vec*>(q);
      } else if constexpr (!EVEN) {
#pragma unroll
        for (int i = 0; i < O::kWide; ++i)
          if (i < left) c[k][i] = q[i];
      }
    }
  }
  // -inf past the end
  __device__ __forceinline__ void get(float (&v)[V], int n) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool has = O::expert(EVEN ? i / O::kWide * O::kWide : i) < n;
      const T e = c[i / O::kWide][i % O::kWide];
      if constexpr (sizeof(T) == 2) v[i] = has ? bf_lo(e) : kNegInf;
      else v[i] = has ? e : kNegInf;
    }
  }
};

template <typename T>
__device__ __forceinline__ float logit_at(const T* row, int e) {
  if constexpr (sizeof(T) == 2) return bf_lo(row[e]);
  else return row[e];
}

// v becomes e^(v - most) with a token's largest logit, most; s: their sum.  False,
// and zeros, for a token of nothing but -inf (one with a NaN, too, has NaNs).
template <int G, int V>
__device__ __forceinline__ bool exponentials(float (&v)[V], float& most, float& s) {
  most = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) most = fmaxf(most, v[i]);
  most = lanes_fmax<G>(most);
  const float by = most == kNegInf ? 0.0f : most;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = weight_of(v[i], by);
    s += v[i];
  }
  s = lanes_sum<G>(s);
  if (s != s) most = s;
  return most != kNegInf;
}

// The `last` (at most 16) next choices of a token, one for each lane to keep; -1
// for none.  key: 0 where taken or not to be chosen.
template <typename T, int G, int V>
__device__ __forceinline__ int choose_exact(uint32_t (&key)[V], int last) {
  using O = Own<T, G, V>;
  const int li = threadIdx.x & (G - 1), at = O::lane();
  int mine = -1;
  for (int j = 0; j < last; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = umax32(best, key[i]);
    best = lanes_max<G>(best);
    int e = 0x4000;  // the lowest expert that has it
#pragma unroll
    for (int i = V - 1; i >= 0; --i) e = key[i] == best ? O::expert(i) : e;
    e = 0x7FFF - (int)lanes_max<G>((uint32_t)(0x7FFF - at - e));
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = e - at == O::expert(i) ? 0 : key[i];
    if (li == j) mine = best ? e : -1;
  }
  return mine;
}

// counts, slope and the part of the loss of an expert with c choices and sum p
__device__ __forceinline__ float settle(const RouteArgs& a, int e, int c, float p, int held) {
  const double n = held;
  const float slope = held ? (float)c * (float)((double)a.experts / (n * n * (double)a.topk)) : 0.0f;
  a.counts[e] = c;
  a.slope[e] = slope;
  return slope * p;
}

template <typename T, int G, int V, bool EVEN, bool CHOSEN>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  constexpr int NT = kRouteThreads, kGroups = NT / G, kWaves = NT / 64;
  constexpr int kAll = G * V;              // experts that there is room for
  constexpr int kBits = log2_of(kAll);     // of an expert's number
  constexpr uint32_t kLow = (1u << kBits) - 1;
  __shared__ int cnt[kAll + 1];
  __shared__ float sums[kWaves][kAll];
  const int tid = threadIdx.x, li = tid & (G - 1), lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= kAll; e += NT) cnt[e] = 0;
  __syncthreads();
  using O = Own<T, G, V>;
  const int at = O::lane(), n = a.experts - at;
  float ps[V];  // sums of p
#pragma unroll
  for (int i = 0; i < V; ++i) ps[i] = 0.0f;
  int held = 0;  // tokens counted
  const T* logits = static_cast<const T*>(a.logits);
  const int tokens = (int)a.tokens, step = a.blocks * kGroups;  // (at most 2^30 tokens)
  const int t_first = blockIdx.x * kGroups + tid / G;
  const bool few = a.topk <= 16;

  Logits<T, G, V, EVEN> next{};
  bool next_real = t_first < tokens && (!a.mask || a.mask[t_first]);
  if (next_real) next.load(logits + t_first * a.ld + at, n);
  // (whole waves go round together: the lanes of a group are never apart)
  for (int t = t_first; __any(t < tokens); t += step) {
    const bool there = t < tokens, real = next_real;
    const T* row = logits + t * a.ld;
    float e[V], most, s;
    uint32_t pk[V];  // (few choices)
    next.get(e, real ? n : 0);
    next_real = t + step < tokens && (!a.mask || a.mask[t + step]);
    if (next_real) next.load(row + step * a.ld + at, n);
    if constexpr (!CHOSEN) {
      uint32_t from_top = kAll - 1 - at;
      asm volatile("" : "+v"(from_top));  // (or V registers would hold the experts' numbers from token to token)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t b = as_bits(e[i] + 0.0f);
        const uint32_t k = __builtin_elementwise_sub_sat(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 0x007FFFFFu);
        pk[i] = ((k & ~kLow) | from_top) ^ (uint32_t)O::expert(i);  // (the expert's number from the top)
      }
    }
    const bool live = exponentials<G, V>(e, most, s);
    const float inv = live ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) ps[i] += e[i] * inv;
    if (live && li == 0) ++held;

    if constexpr (CHOSEN) {
      if (live)
        for (int j = li; j < a.topk; j += G) {
          int64_t x;
          if (a.wide) x = static_cast<const int64_t*>(a.chosen)[t * a.ld_chosen + j];
          else x = static_cast<const int32_t*>(a.chosen)[t * a.ld_chosen + j];
          if (x >= 0 && x < a.experts) atomicAdd(&cnt[x], 1);
        }
    } else {
      int mine = -1;  // this lane's choice of the first 16
      bool again = !few;
      if (few) {
        uint32_t best = pk[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = umax32(best, pk[i]);
        best = lanes_max<G>(best);
        bool odd = s != s;
        for (int j = 0; j < a.topk; ++j) {
          if (li == j) mine = (int)(~best & kLow);
          odd = odd || best <= kLow;
          if (sizeof(T) == 2 && j + 1 == a.topk) break;  // (BF16: what was cut off is zero)
          uint32_t other = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) other = umax32(other, pk[i] - best);
          other = lanes_max<G>(other) + best;
          if (sizeof(T) == 4) odd = odd || (other ^ best) <= kLow;
          best = other;
        }
        again = __any(odd && live);
      }
      const int slot = t * a.topk;
      if (again) {
        Logits<T, G, V, EVEN> raw{};
        float v[V];
        uint32_t key[V];
        if (real) raw.load(row + at, n);
        raw.get(v, real ? n : 0);
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(v[i]);
        if (few) {
          mine = choose_exact<T, G, V>(key, a.topk);
        } else {
          for (int base = 0; base < a.topk; base += 16) {
            mine = choose_exact<T, G, V>(key, min(a.topk - base, 16));
            if (there && li < 16 && base + li < a.topk) a.expert[slot + base + li] = mine;
          }
        }
      }
      // weights: few choices are one to a lane, others were just written by it
      float total = 0.0f;
      if (few) {
        float w = 0.0f;
        const bool has = live && li < a.topk && mine >= 0;
        if (has) {
          atomicAdd(&cnt[mine], 1);
          w = weight_of(logit_at(row, mine), most);
        }
        if (a.normalize) total = lanes_sum<G>(w);
        if (there && li < a.topk) {
          a.expert[slot + li] = has ? mine : -1;
          a.weights[slot + li] = !has ? 0.0f : w / (a.normalize ? total : s);
        }
      } else {
        for (int pass = a.normalize ? 0 : 1; pass < 2; ++pass) {
          const float by = a.normalize ? total : s;
          if (there && li < 16)
            for (int j = li; j < a.topk; j += 16) {
              const int x = a.expert[slot + j];
              const float w = x >= 0 ? weight_of(logit_at(row, x), most) : 0.0f;
              if (pass == 0) {
                total += w;
              } else {
                a.weights[slot + j] = x >= 0 ? w / by : 0.0f;
                if (x >= 0) atomicAdd(&cnt[x], 1);
              }
            }
          if (pass == 0) total = lanes_sum<G>(total);
        }
      }
    }
  }

  // the workgroup's sums: the groups of a wave, then the waves
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (G == 16) {
      ps[i] += __shfl_xor(ps[i], 16, 64);
      ps[i] += __shfl_xor(ps[i], 32, 64);
    }
    if (lane < G) sums[wave][at + O::expert(i)] = ps[i];
  }
  if (li == 0 && held) atomicAdd(&cnt[kAll], held);
  __syncthreads();
  auto sum_of = [&](int e) {
    float p = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) p += sums[w][e];
    return p;
  };
  if (a.blocks == 1) {  // all there is
    __shared__ float parts[kWaves];
    float loss = 0.0f;
    for (int e = tid; e < a.experts; e += NT) loss += settle(a, e, cnt[e], sum_of(e), cnt[kAll]);
    loss = wave_sum(loss);
    if (lane == 0) parts[wave] = loss;
    __syncthreads();
    if (tid == 0) {
      loss = 0.0f;
      for (int w = 0; w < kWaves; ++w) loss += parts[w];
      *a.loss = loss;
    }
    return;
  }
  for (int e = tid; e < a.experts; e += NT) {
    a.psum[(int64_t)blockIdx.x * a.experts + e] = sum_of(e);
    a.hist[(int64_t)blockIdx.x * a.experts + e] = cnt[e];
  }
  if (tid == 0) {
    a.held[blockIdx.x] = cnt[kAll];
    if (blockIdx.x == 0) *a.ticket = 0;
  }
}

// Counts, slope and loss from the workgroups' sums: a workgroup takes 32 experts,
// each of its 32 thread groups every 32nd sum; the last one to end adds up the
// parts of the loss, in order.
constexpr int kSumThreads = 1024, kSumExperts = 32, kSumGroups = kSumThreads / kSumExperts;
__global__ __launch_bounds__(kSumThreads) void route_sum_kernel(RouteArgs a) {
  __shared__ int c_part[kSumGroups][kSumExperts + 1];
  __shared__ float p_part[kSumGroups][kSumExperts + 1];
  __shared__ int tokens[kSumThreads / 64];
  __shared__ float parts[kSumExperts];
  const int tid = threadIdx.x, x = tid & (kSumExperts - 1), g = tid / kSumExperts;
  const int first = (int)blockIdx.x * kSumExperts;
  int c = 0, n = tid < a.blocks ? a.held[tid] : 0;
  float p = 0.0f;
  constexpr int kMost = kRouteMaxBlocks / kSumGroups;
  int cs[kMost];
  float pq[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int b = g + i * kSumGroups;
    const bool has = b < a.blocks && first + x < a.experts;
    cs[i] = has ? a.hist[(int64_t)b * a.experts + first + x] : 0;
    pq[i] = has ? a.psum[(int64_t)b * a.experts + first + x] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    c += cs[i];
    p += pq[i];
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, 64);
  if ((tid & 63) == 0) tokens[tid >> 6] = n;
  c_part[g][x] = c;
  p_part[g][x] = p;
  __syncthreads();
  // from here on 32 lanes have an expert: its sums by group
  c = c_part[x][g];
  p = p_part[x][g];
#pragma unroll
  for (int off = kSumGroups / 2; off > 0; off >>= 1) {
    c += __shfl_xor(c, off, 64);
    p += __shfl_xor(p, off, 64);
  }
  if (x == 0) {
    n = 0;
#pragma unroll
    for (int w = 0; w < kSumThreads / 64; ++w) n += tokens[w];
    parts[g] = first + g < a.experts ? settle(a, first + g, c, p, n) : 0.0f;
  }
  __syncthreads();
  if (tid >= 64) return;
  float loss = wave_sum(tid < kSumExperts ? parts[tid] : 0.0f);
  if (tid != 0) return;
  if (gridDim.x > 1) {
    a.part[blockIdx.x] = loss;
    __threadfence();
    if (atomicAdd(a.ticket, 1u) != gridDim.x - 1) return;
    __threadfence();
    loss = 0.0f;
    for (unsigned b = 0; b < gridDim.x; ++b) loss += __hip_atomic_load(a.part + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  *a.loss = loss;
}

// The logits' gradient: the same lanes to a token.  What the weights add falls on
// the topk chosen experts: each lane has a choice and adds it to a row in LDS
// that is zero otherwise, and from which the lanes take their experts' parts.
// 4 workgroups per compute unit: what one sets up is used for more tokens (65536 x
// 256 FP32: 31 us; 2 37, 8 34, 16 37).
constexpr int kBackThreads = 256, kBackBlocks = 4;

template <typename T, int G, int V, bool EVEN>
__global__ __launch_bounds__(kBackThreads) void route_backward_kernel(RouteArgs a) {
  constexpr int kGroups = kBackThreads / G;
  __shared__ __attribute__((aligned(16))) float adds[kGroups][G * V];
  using O = Own<T, G, V>;
  const int tid = threadIdx.x, li = tid & (G - 1), at = O::lane(), n = a.experts - at;
  float* add = adds[tid / G];
  float slope[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    slope[i] = 0.0f;
    add[at + O::expert(i)] = 0.0f;
  }
  if (a.dloss) {
    // What all slopes have in common (all of it, with even loads) has no gradient: it
    // is taken out before anything is rounded to its size.
    const float d = *a.dloss;
    float least = kNegInf;  // (of their negatives the largest)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (O::expert(i) < n) {
        slope[i] = a.slope[at + O::expert(i)];
        least = fmaxf(least, -slope[i]);
      }
    least = fmaxf(-lanes_fmax<G>(least), 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (O::expert(i) < n) slope[i] = d * (slope[i] - least);
  }
  const int tokens = (int)a.tokens, step = (int)gridDim.x * kGroups;  // (at most 2^30 tokens)
  Logits<T, G, V, EVEN> raw{};
  for (int t = (int)blockIdx.x * kGroups + tid / G; __any(t < tokens); t += step) {
    const bool there = t < tokens;
    const bool real = there && (!a.mask || a.mask[t]);
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const int slot = t * a.topk;
    if (real) raw.load(row + at, n);
    int mine = -1;  // the lane's first choice and its gradient
    float dw = 0.0f, chosen = 0.0f;
    if (a.dweights && real && li < a.topk) {
      mine = a.expert[slot + li];
      dw = a.dweights[slot + li];
      if ((unsigned)mine < (unsigned)a.experts) chosen = logit_at(row, mine);
      else mine = -1;
    }
    float v[V], most, s, dot = 0.0f;
    raw.get(v, real ? n : 0);
    const bool live = exponentials<G, V>(v, most, s);
#pragma unroll
    for (int i = 0; i < V; ++i) dot += v[i] * slope[i];
    dot = lanes_sum<G>(dot);
    const float inv = live ? 1.0f / s : 0.0f;
    dot *= inv;

    if (a.dweights) {
      // the choices' e^, their sum and that of e^ dw
      const float w = mine >= 0 ? weight_of(chosen, most) : 0.0f;
      float total = w, along = w * dw;
      if (mine < 0) along = 0.0f;
      if (a.topk > G && real)
        for (int j = li + G; j < a.topk; j += G) {
          const int e = a.expert[slot + j];
          if ((unsigned)e < (unsigned)a.experts) {
            const float x = weight_of(logit_at(row, e), most);
            total += x;
            along += x * a.dweights[slot + j];
          }
        }
      along = lanes_sum<G>(along);
      float unit = inv;  // e^ to weight
      if (a.normalize) {
        total = lanes_sum<G>(total);
        unit = live && total != 0.0f ? 1.0f / total : 0.0f;
      }
      along *= unit;
      if (!a.normalize) dot += along;
      const float less = a.normalize ? along : 0.0f;
      float rest = 0.0f;
      if (a.normalize) {
        // <w, dw - less> is what less is off by, which is all there is of dw - less
        // where one expert has nearly all the weight: it is taken out, too
        if (mine >= 0) rest = w * unit * (dw - less);
        if (a.topk > G && real)
          for (int j = li + G; j < a.topk; j += G) {
            const int e = a.expert[slot + j];
            if ((unsigned)e < (unsigned)a.experts)
              rest += weight_of(logit_at(row, e), most) * unit * (a.dweights[slot + j] - less);
          }
        rest = lanes_sum<G>(rest);
      }
      if (mine >= 0) atomicAdd(add + mine, w * unit * (dw - less - rest));
      if (a.topk > G && real)
        for (int j = li + G; j < a.topk; j += G) {
          const int e = a.expert[slot + j];
          if ((unsigned)e < (unsigned)a.experts)
            atomicAdd(add + e, weight_of(logit_at(row, e), most) * unit * (a.dweights[slot + j] - less - rest));
        }
      // (the group's lanes are in one wave, whose LDS operations stay in order)
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = v[i] * inv * (slope[i] - dot);
      if (a.dweights) v[i] += add[at + O::expert(i)];
      if (!live) v[i] = 0.0f;
    }
    if (a.dweights) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (mine >= 0) add[mine] = 0.0f;
      if (a.topk > G) {
#pragma unroll
        for (int i = 0; i < V; ++i) add[at + O::expert(i)] = 0.0f;
      }
    }
    if (there) {
      T* out = static_cast<T*>(a.dlogits) + t * a.ld_dlogits + at;
#pragma unroll
      for (int c = 0; c < V; c += O::kWide) {
        T o[O::kWide];
#pragma unroll
        for (int i = 0; i < O::kWide; ++i) {
          if constexpr (sizeof(T) == 2) o[i] = __builtin_bit_cast(uint16_t, (__bf16)v[c + i]);
          else o[i] = v[c + i];
        }
        const int left = n - O::expert(c);
        if constexpr (O::kWide == 1) {
          if (left > 0) out[O::expert(c)] = o[0];
        } else if (EVEN ? left > 0 : left >= O::kWide) {
          typename O::vec x;
#pragma unroll
          for (int i = 0; i < O::kWide; ++i) x[i] = o[i];
          *reinterpret_cast<typename O::vec*>(out + O::expert(c)) = x;
        } else if constexpr (!EVEN) {
#pragma unroll
          for (int i = 0; i < O::kWide; ++i)
            if (i < left) out[O::expert(c) + i] = o[i];
        }
      }
    }
  }
}

RouteArgs args_of(const RouteParams& p) {
  RouteArgs a{};
  a.logits = p.logits;
  a.tokens = p.tokens;
  a.ld = p.ld;
  a.experts = (int)p.experts;
  a.topk = (int)p.topk;
  a.normalize = p.normalize;
  a.mask = p.mask;
  a.expert = p.expert;
  a.weights = p.weights;
  a.chosen = p.chosen;
  a.wide = p.idx_dtype == 1;
  a.ld_chosen = p.ld_chosen;
  a.loss = p.loss;
  a.counts = p.counts;
  a.slope = p.slope;
  a.blocks = (int)route_blocks(p.tokens, p.experts);
  a.psum = static_cast<float*>(p.workspace);
  if (a.blocks > 1) {
    a.hist = reinterpret_cast<int32_t*>(a.psum + a.blocks * p.experts);
    a.held = a.hist + a.blocks * p.experts;
    a.part = reinterpret_cast<float*>(a.held + a.blocks);
    a.ticket = reinterpret_cast<uint32_t*>(a.part + kMaxExperts / kSumExperts);
  }
  a.dweights = p.dweights;
  a.dloss = p.dloss;
  a.dlogits = p.dlogits;
  a.ld_dlogits = p.ld_dlogits;
  return a;
}

template <typename T, int G, int V, bool EVEN>
hipError_t route(const RouteArgs& a, bool given, hipStream_t st) {
  if (given) route_kernel<T, G, V, EVEN, true><<<(unsigned)a.blocks, kRouteThreads, 0, st>>>(a);
  else route_kernel<T, G, V, EVEN, false><<<(unsigned)a.blocks, kRouteThreads, 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.blocks == 1) return e;
  route_sum_kernel<<<(unsigned)((a.experts + kSumExperts - 1) / kSumExperts), kSumThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int G, int V, bool EVEN>
hipError_t route_back(const RouteArgs& a, hipStream_t st) {
  constexpr int kGroups = kBackThreads / G;
  const int64_t need = (a.tokens + kGroups - 1) / kGroups, most = kBackBlocks * (int64_t)cu_count(stream_device(st));
  route_backward_kernel<T, G, V, EVEN><<<(unsigned)(need < most ? need : most), kBackThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool BACK>
hipError_t route_any(const RouteArgs& a, bool given, hipStream_t st) {
  auto go = [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    const bool even = a.experts % Own<T, G, V>::kWide == 0;
    if constexpr (BACK) return even ? route_back<T, G, V, true>(a, st) : route_back<T, G, V, false>(a, st);
    else return even ? route<T, G, V, true>(a, given, st) : route<T, G, V, false>(a, given, st);
  };
  const std::integral_constant<int, 16> row;
  const std::integral_constant<int, 64> wave;
  const std::integral_constant<int, 8> v8;
  const std::integral_constant<int, 16> v16;
  switch (per_lane(a.experts)) {
    case 1: return go(row, std::integral_constant<int, 1>{});
    case 2: return go(row, std::integral_constant<int, 2>{});
    case 4: return go(row, std::integral_constant<int, 4>{});
    case 8: return lanes_of(a.experts) == 16 ? go(row, v8) : go(wave, v8);
  }
  return lanes_of(a.experts) == 16 ? go(row, v16) : go(wave, v16);
}

}  // namespace

// workgroups of the forward pass
int64_t route_blocks(int64_t tokens, int64_t experts) {
  const int64_t groups = kRouteThreads / lanes_of(experts);
  if (tokens <= kRouteOneBlock * groups) return 1;
  const int64_t n = (tokens + groups - 1) / groups;
  return n < kRouteMaxBlocks ? n : kRouteMaxBlocks;
}

// bytes that they leave for the second launch (none where there is one)
int64_t route_workspace(int64_t tokens, int64_t experts) {
  const int64_t blocks = route_blocks(tokens, experts);
  return blocks > 1 ? (blocks * (2 * experts + 1) + kMaxExperts / kSumExperts + 1) * (int64_t)sizeof(float) : 0;
}

hipError_t launch_route(const RouteParams& p, hipStream_t st) {
  const RouteArgs a = args_of(p);
  return p.dtype == kInBf16 ? route_any<uint16_t, false>(a, p.given, st) : route_any<float, false>(a, p.given, st);
}

hipError_t launch_route_backward(const RouteParams& p, hipStream_t st) {
  const RouteArgs a = args_of(p);
  return p.dtype == kInBf16 ? route_any<uint16_t, true>(a, false, st) : route_any<float, true>(a, false, st);
}

}  // namespace fp8mi
