// route.hip -- the experts' router for gfx950: softmax over the experts, the
// choice of the topk largest, their weights, the slots of each expert and the
// balance loss, with the logits' gradient.
//
//   p = softmax(l), loss = experts sum_e f_e P_e,
//   f_e = counts_e / (n topk), P_e = sum over tokens of p_te / n, n tokens,
//   slope_e = d loss / d p_te = experts f_e / n (the counts have no gradient),
//   dp = dloss slope + (the weights' part), dl = p (dp - <p, dp>).
//
// 16 lanes own a token, V neighbouring experts each, so that a maximum or a sum
// over the experts is one of V registers and four DPP rotations; the next
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
#include "launch.hpp"
#include "rows.hpp"
#include "tile.hpp"

namespace fp8mi {

namespace {

constexpr int kRouteMaxBlocks = 256;
constexpr int kRouteOneBlock = 4;  // tokens per group of lanes up to which there is one workgroup, and one launch

// threads of the forward pass: as many as the registers of V experts allow
constexpr int route_threads(int v) { return v <= 16 ? 1024 : (v <= 32 ? 512 : 256); }
// experts per lane: the power of two that 16 lanes hold them with
constexpr int per_lane(int64_t experts) {
  int v = 1;
  while (16 * v < experts) v *= 2;
  return v;
}
constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

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

__device__ __forceinline__ float row16_sum(float v) {
  v += as_float(dpp<0x128>(as_bits(v)));
  v += as_float(dpp<0x124>(as_bits(v)));
  v += as_float(dpp<0x122>(as_bits(v)));
  return v + as_float(dpp<0x121>(as_bits(v)));
}
__device__ __forceinline__ float row16_fmax(float v) {
  v = fmaxf(v, as_float(dpp<0x128>(as_bits(v))));
  v = fmaxf(v, as_float(dpp<0x124>(as_bits(v))));
  v = fmaxf(v, as_float(dpp<0x122>(as_bits(v))));
  return fmaxf(v, as_float(dpp<0x121>(as_bits(v))));
}

constexpr float kNegInf = -__builtin_inff();

// an integer that orders like the logit, NaN on top; 0: not to be chosen (-inf)
__device__ __forceinline__ uint32_t key_of(float v) {
  v += 0.0f;  // -0 is 0
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = as_bits(v);
  return __builtin_elementwise_sub_sat(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 0x007FFFFFu);
}

// e^(v - most)
__device__ __forceinline__ float weight_of(float v, float most) {
  return __builtin_amdgcn_exp2f((v - most) * 1.44269504088896340736f);
}

// V logits as they lie in memory, of which n are there.  EVEN: the number of
// experts is a multiple of V, or of 8, so that no vector is cut.
template <typename T, int V, bool EVEN>
struct Logits {
  static constexpr int kChunks = V >= 8 ? V / 8 : 1;
  typedef T vec __attribute__((ext_vector_type(V == 4 ? 4 : 2), aligned(sizeof(T))));
  Chunk<T> c[kChunks];
  T e[V >= 8 ? 1 : V];
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (V >= 8) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        if constexpr (EVEN) {
          if (n > 8 * k) c[k].load(p + 8 * k, 8);
        } else {
          c[k].load(p + 8 * k, n - 8 * k);
        }
      }
    } else if constexpr (V == 1) {
      if (n > 0) e[0] = p[0];
    } else {
      if (EVEN ? n > 0 : n >= V) {
        const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = v[i];
      } else if constexpr (!EVEN) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < n) e[i] = p[i];
      }
    }
  }
  // -inf past the end
  __device__ __forceinline__ void get(float (&v)[V], int n) const {
    if constexpr (V >= 8) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        float w[8];
        c[k].get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * k + i] = (EVEN ? 8 * k : 8 * k + i) < n ? w[i] : kNegInf;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (sizeof(T) == 2) v[i] = (EVEN ? 0 : i) < n ? bf_lo(e[i]) : kNegInf;
        else v[i] = (EVEN ? 0 : i) < n ? e[i] : kNegInf;
      }
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
template <int V>
__device__ __forceinline__ bool exponentials(float (&v)[V], float& most, float& s) {
  most = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) most = fmaxf(most, v[i]);
  most = row16_fmax(most);
  const float by = most == kNegInf ? 0.0f : most;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = weight_of(v[i], by);
    s += v[i];
  }
  s = row16_sum(s);
  if (s != s) most = s;
  return most != kNegInf;
}

// The `last` (at most 16) next choices of a token, one for each lane to keep; -1
// for none.  key: 0 where taken or not to be chosen.
template <int V>
__device__ __forceinline__ int choose_exact(uint32_t (&key)[V], int last) {
  const int li = threadIdx.x & 15, at = li * V;
  int mine = -1;
  for (int j = 0; j < last; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = umax32(best, key[i]);
    best = row16_max(best);
    int e = 0x4000;  // the lowest expert that has it
#pragma unroll
    for (int i = V - 1; i >= 0; --i) e = key[i] == best ? i : e;
    e = 0x7FFF - (int)row16_max((uint32_t)(0x7FFF - at - e));
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = e - at == i ? 0 : key[i];
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

template <typename T, int V, bool EVEN, bool CHOSEN>
__global__ __launch_bounds__(route_threads(V)) void route_kernel(RouteArgs a) {
  constexpr int NT = route_threads(V), kGroups = NT / 16, kWaves = NT / 64;
  constexpr int kBits = log2_of(16 * V);  // of an expert's number
  constexpr uint32_t kLow = (1u << kBits) - 1;
  __shared__ int cnt[16 * V + 1];
  __shared__ float sums[kWaves][16 * V];
  const int tid = threadIdx.x, li = tid & 15, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= 16 * V; e += NT) cnt[e] = 0;
  __syncthreads();
  const int at = li * V, n = a.experts - at;  // this lane's experts, of which n are there
  float ps[V];                                // sums of p
#pragma unroll
  for (int i = 0; i < V; ++i) ps[i] = 0.0f;
  int held = 0;  // tokens counted
  const T* logits = static_cast<const T*>(a.logits);
  const int tokens = (int)a.tokens, step = a.blocks * kGroups;  // (at most 2^30 tokens)
  const int t_first = blockIdx.x * kGroups + (tid >> 4);
  const bool few = a.topk <= 16;

  Logits<T, V, EVEN> next;
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
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t b = as_bits(e[i] + 0.0f);
        const uint32_t k = __builtin_elementwise_sub_sat(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 0x007FFFFFu);
        pk[i] = ((k & ~kLow) | (uint32_t)(16 * V - 1 - at)) ^ (uint32_t)i;  // (the expert's number from the top)
      }
    }
    const bool live = exponentials<V>(e, most, s);
    const float inv = live ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) ps[i] += e[i] * inv;
    if (live && li == 0) ++held;

    if constexpr (CHOSEN) {
      if (live)
        for (int j = li; j < a.topk; j += 16) {
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
        best = row16_max(best);
        bool odd = s != s;
        for (int j = 0; j < a.topk; ++j) {
          if (li == j) mine = (int)(~best & kLow);
          odd = odd || best <= kLow;
          if (sizeof(T) == 2 && j + 1 == a.topk) break;  // (BF16: what was cut off is zero)
          uint32_t other = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) other = umax32(other, pk[i] - best);
          other = row16_max(other) + best;
          if (sizeof(T) == 4) odd = odd || (other ^ best) <= kLow;
          best = other;
        }
        again = __any(odd && live);
      }
      const int slot = t * a.topk;
      if (again) {
        Logits<T, V, EVEN> raw;
        float v[V];
        uint32_t key[V];
        if (real) raw.load(row + at, n);
        raw.get(v, real ? n : 0);
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = key_of(v[i]);
        if (few) {
          mine = choose_exact<V>(key, a.topk);
        } else {
          for (int base = 0; base < a.topk; base += 16) {
            mine = choose_exact<V>(key, min(a.topk - base, 16));
            if (there && base + li < a.topk) a.expert[slot + base + li] = mine;
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
        if (a.normalize) total = row16_sum(w);
        if (there && li < a.topk) {
          a.expert[slot + li] = has ? mine : -1;
          a.weights[slot + li] = !has ? 0.0f : (a.normalize ? w / total : w * inv);
        }
      } else {
        for (int pass = a.normalize ? 0 : 1; pass < 2; ++pass) {
          const float by = a.normalize ? 1.0f / total : inv;
          if (there)
            for (int j = li; j < a.topk; j += 16) {
              const int x = a.expert[slot + j];
              const float w = x >= 0 ? weight_of(logit_at(row, x), most) : 0.0f;
              if (pass == 0) {
                total += w;
              } else {
                a.weights[slot + j] = x >= 0 ? w * by : 0.0f;
                if (x >= 0) atomicAdd(&cnt[x], 1);
              }
            }
          if (pass == 0) total = row16_sum(total);
        }
      }
    }
  }

  // the workgroup's sums: the four groups of a wave, then the waves
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ps[i] += __shfl_xor(ps[i], 16, 64);
    ps[i] += __shfl_xor(ps[i], 32, 64);
    if (lane < 16) sums[wave][at + i] = ps[i];
  }
  if (li == 0 && held) atomicAdd(&cnt[16 * V], held);
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
    for (int e = tid; e < a.experts; e += NT) loss += settle(a, e, cnt[e], sum_of(e), cnt[16 * V]);
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
    a.held[blockIdx.x] = cnt[16 * V];
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
constexpr int kBackThreads = 256, kBackGroups = kBackThreads / 16;

template <typename T, int V, bool EVEN>
__global__ __launch_bounds__(kBackThreads) void route_backward_kernel(RouteArgs a) {
  __shared__ __attribute__((aligned(16))) float adds[kBackGroups][16 * V];
  const int tid = threadIdx.x, li = tid & 15, at = li * V, n = a.experts - at;
  float* add = adds[tid >> 4];
  float slope[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    slope[i] = 0.0f;
    add[at + i] = 0.0f;
  }
  if (a.dloss) {
    const float d = *a.dloss;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) slope[i] = d * a.slope[at + i];
  }
  const int tokens = (int)a.tokens, step = (int)gridDim.x * kBackGroups;  // (at most 2^30 tokens)
  for (int t = (int)blockIdx.x * kBackGroups + (tid >> 4); __any(t < tokens); t += step) {
    const bool there = t < tokens;
    const bool real = there && (!a.mask || a.mask[t]);
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    const int slot = t * a.topk;
    Logits<T, V, EVEN> raw;
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
    const bool live = exponentials<V>(v, most, s);
#pragma unroll
    for (int i = 0; i < V; ++i) dot += v[i] * slope[i];
    dot = row16_sum(dot);
    const float inv = live ? 1.0f / s : 0.0f;
    dot *= inv;

    if (a.dweights) {
      // the choices' e^, their sum and that of e^ dw
      const float w = mine >= 0 ? weight_of(chosen, most) : 0.0f;
      float total = w, along = w * dw;
      if (mine < 0) along = 0.0f;
      if (a.topk > 16 && real)
        for (int j = li + 16; j < a.topk; j += 16) {
          const int e = a.expert[slot + j];
          if ((unsigned)e < (unsigned)a.experts) {
            const float x = weight_of(logit_at(row, e), most);
            total += x;
            along += x * a.dweights[slot + j];
          }
        }
      along = row16_sum(along);
      float unit = inv;  // e^ to weight
      if (a.normalize) {
        total = row16_sum(total);
        unit = live && total != 0.0f ? 1.0f / total : 0.0f;
      }
      along *= unit;
      if (!a.normalize) dot += along;
      const float less = a.normalize ? along : 0.0f;
      if (mine >= 0) atomicAdd(add + mine, w * unit * (dw - less));
      if (a.topk > 16 && real)
        for (int j = li + 16; j < a.topk; j += 16) {
          const int e = a.expert[slot + j];
          if ((unsigned)e < (unsigned)a.experts)
            atomicAdd(add + e, weight_of(logit_at(row, e), most) * unit * (a.dweights[slot + j] - less));
        }
      // (the group's lanes are in one wave, whose LDS operations stay in order)
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = v[i] * inv * (slope[i] - dot);
      if (a.dweights) v[i] += add[at + i];
      if (!live) v[i] = 0.0f;
    }
    if (a.dweights) {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (mine >= 0) add[mine] = 0.0f;
      if (a.topk > 16) {
#pragma unroll
        for (int i = 0; i < V; ++i) add[at + i] = 0.0f;
      }
    }
    if (there) {
      T* out = static_cast<T*>(a.dlogits) + t * a.ld_dlogits + at;
      if constexpr (V >= 8) {
#pragma unroll
        for (int c = 0; c < V / 8; ++c) {
          Chunk<T> k;
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = v[8 * c + e];
          k.set(w);
          if constexpr (EVEN) {
            if (n > 8 * c) k.store(out + 8 * c, 8);
          } else {
            k.store(out + 8 * c, n - 8 * c);
          }
        }
      } else {
        T o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if constexpr (sizeof(T) == 2) o[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
          else o[i] = v[i];
        }
        if constexpr (EVEN && V > 1) {
          typename Logits<T, V, EVEN>::vec x;
#pragma unroll
          for (int i = 0; i < V; ++i) x[i] = o[i];
          if (n > 0) *reinterpret_cast<typename Logits<T, V, EVEN>::vec*>(out) = x;
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < n) out[i] = o[i];
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

template <typename T, int V, bool EVEN>
hipError_t route(const RouteArgs& a, bool given, hipStream_t st) {
  if (given) route_kernel<T, V, EVEN, true><<<(unsigned)a.blocks, route_threads(V), 0, st>>>(a);
  else route_kernel<T, V, EVEN, false><<<(unsigned)a.blocks, route_threads(V), 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.blocks == 1) return e;
  route_sum_kernel<<<(unsigned)((a.experts + kSumExperts - 1) / kSumExperts), kSumThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int V, bool EVEN>
hipError_t route_back(const RouteArgs& a, hipStream_t st) {
  const int64_t groups = (a.tokens + kBackGroups - 1) / kBackGroups, most = 8 * (int64_t)cu_count(stream_device(st));
  route_backward_kernel<T, V, EVEN><<<(unsigned)(groups < most ? groups : most), kBackThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, bool BACK>
hipError_t route_any(const RouteArgs& a, bool given, hipStream_t st) {
  auto go = [&](auto v) {
    constexpr int V = decltype(v)::value;
    const bool even = a.experts % (V < 8 ? V : 8) == 0;
    if constexpr (BACK) return even ? route_back<T, V, true>(a, st) : route_back<T, V, false>(a, st);
    else return even ? route<T, V, true>(a, given, st) : route<T, V, false>(a, given, st);
  };
  switch (per_lane(a.experts)) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
  }
  return go(std::integral_constant<int, 64>{});
}

}  // namespace

// workgroups of the forward pass
int64_t route_blocks(int64_t tokens, int64_t experts) {
  const int64_t groups = route_threads(per_lane(experts)) / 16;
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
