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
// over the experts is one of V registers and four DPP rotations, and equal
// logits are in the order of the lanes.  Logits are compared as integers that
// order like them (NaN on top, -0 with 0); an expert of logit -inf, and one that
// is taken, has the integer 0 and is not chosen.  Sums over the tokens are
// taken in registers, then over the workgroup and, by a second launch in a fixed
// order, over all workgroups; only integers are counted with atomics.
#include <atomic>

#include "launch.hpp"
#include "rows.hpp"
#include "tile.hpp"

namespace fp8mi {

namespace {

constexpr int kRouteThreads = 256, kRouteGroups = kRouteThreads / 16;
constexpr int kRouteMaxBlocks = 512;
constexpr int kRouteTokens = 4;  // tokens per group of lanes before there are more workgroups

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
  float* psum;    // [blocks][experts]
  int32_t* hist;  // [blocks][experts + 1], the last one tokens
  const float* dweights;
  const float* dloss;
  void* dlogits;
  int64_t ld_dlogits;
};

__device__ __forceinline__ float row16_sum(float v) {
  auto add = [](float x, uint32_t o) __attribute__((always_inline)) { return x + __builtin_bit_cast(float, o); };
  v = add(v, dpp<0x128>(__builtin_bit_cast(uint32_t, v)));
  v = add(v, dpp<0x124>(__builtin_bit_cast(uint32_t, v)));
  v = add(v, dpp<0x122>(__builtin_bit_cast(uint32_t, v)));
  return add(v, dpp<0x121>(__builtin_bit_cast(uint32_t, v)));
}

// an integer that orders like the logit; 0: not to be chosen
__device__ __forceinline__ uint32_t key_of(float v) {
  v += 0.0f;  // -0 is 0
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const uint32_t k = (int32_t)b < 0 ? ~b : b | 0x80000000u;
  return k == 0x007FFFFFu ? 0u : k;  // -inf
}
__device__ __forceinline__ float logit_of(uint32_t k) {
  if (k == 0) return -__builtin_inff();
  return __builtin_bit_cast(float, (k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);  // (NaN stays NaN)
}

// V logits of a token from expert `at` on, as integers (0 past the end)
template <typename T, int V>
__device__ __forceinline__ void load_logits(float (&v)[V], const T* p, int at, int experts) {
  if constexpr (V >= 8) {
#pragma unroll
    for (int c = 0; c < V / 8; ++c) {
      Chunk<T> k;
      float w[8];
      const int n = experts - at - 8 * c;
      k.load(p + at + 8 * c, n);
      k.get(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * c + e] = e < n ? w[e] : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (at + e < experts) {
        if constexpr (sizeof(T) == 2) v[e] = bf_lo(p[at + e]);
        else v[e] = p[at + e];
      } else {
        v[e] = -__builtin_inff();
      }
    }
  }
}

// e^(v - most) of the experts, 0 for -inf (whose token has another)
__device__ __forceinline__ float weight_of(float v, float most) { return __expf(v - most); }

template <typename T, int V, bool CHOSEN>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  __shared__ int cnt[kMaxExperts + 1];
  __shared__ float sums[4][16 * V];
  const int tid = threadIdx.x, li = tid & 15, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= a.experts; e += kRouteThreads) cnt[e] = 0;
  __syncthreads();
  const int at = li * V;
  float ps[V];  // sums of p
#pragma unroll
  for (int i = 0; i < V; ++i) ps[i] = 0.0f;
  int held = 0;  // tokens counted

  // (whole waves go round together: the lanes of a group are never apart)
  for (int64_t t0 = (int64_t)blockIdx.x * kRouteGroups; t0 < a.tokens; t0 += (int64_t)a.blocks * kRouteGroups) {
    const int64_t t = t0 + (tid >> 4);
    const bool there = t < a.tokens;
    const bool real = there && (!a.mask || a.mask[t]);
    float v[V];
    uint32_t key[V], top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = -__builtin_inff();
    if (real) load_logits<T, V>(v, static_cast<const T*>(a.logits) + t * a.ld, at, a.experts);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = key_of(v[i]);
      top = umax32(top, key[i]);
    }
    top = row16_max(top);
    const float most = logit_of(top);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = top == 0 ? 0.0f : weight_of(v[i], most);
      s += v[i];
    }
    s = row16_sum(s);
    const float inv = top == 0 ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < V; ++i) ps[i] += v[i] * inv;
    if (top != 0 && li == 0) ++held;

    if constexpr (CHOSEN) {
      if (real && top != 0)
        for (int j = li; j < a.topk; j += 16) {
          int64_t e;
          if (a.wide) e = static_cast<const int64_t*>(a.chosen)[t * a.ld_chosen + j];
          else e = static_cast<const int32_t*>(a.chosen)[t * a.ld_chosen + j];
          if (e >= 0 && e < a.experts) atomicAdd(&cnt[e], 1);
        }
    } else {
      float total = 0.0f;  // of the chosen ones' e^
      for (int base = 0; base < a.topk; base += 16) {
        // the choices base .. base + 15: one for each lane to keep
        int mine = -1;
        float mine_w = 0.0f;
        const int last = min(a.topk - base, 16);
        for (int j = 0; j < last; ++j) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) m = umax32(m, key[i]);
          const uint32_t best = row16_max(m);
          // the lowest lane that has it, and in it the lowest expert
          const uint64_t has = __ballot(m == best && best != 0);
          const uint32_t group = (uint32_t)(has >> (lane & 48)) & 0xFFFFu;
          const int win = __ffs((int)group) - 1;
          int e = -1;
          float w = 0.0f;
          if (li == win) {
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
              if (key[i] == best) {
                e = at + i;
                w = v[i];
              }
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (at + i == e) key[i] = 0;
            atomicAdd(&cnt[e], 1);
          }
          const int from = win < 0 ? lane : (lane & 48) | win;
          e = __shfl(e, from, 64);
          w = __shfl(w, from, 64);
          if (win < 0) e = -1;
          if (li == j) {
            mine = e;
            mine_w = e < 0 ? 0.0f : w;
          }
        }
        if (there && li < last) a.expert[t * a.topk + base + li] = mine;
        total += row16_sum(mine_w);
        if (!a.normalize || a.topk <= 16) {
          if (there && li < last)
            a.weights[t * a.topk + base + li] = mine < 0 ? 0.0f : (a.normalize ? mine_w / total : mine_w * inv);
        } else if (there && li < last) {
          a.weights[t * a.topk + base + li] = mine_w;
        }
      }
      if (a.normalize && a.topk > 16 && there) {
        for (int j = li; j < a.topk; j += 16) {
          float* w = a.weights + t * a.topk + j;  // (this lane's own)
          *w = total == 0.0f ? 0.0f : *w / total;
        }
      }
    }
  }

  // the workgroup's sums: the four groups of a wave, then the waves
#pragma unroll
  for (int i = 0; i < V; ++i) {
    ps[i] += __shfl_xor(ps[i], 16, 64);
    ps[i] += __shfl_xor(ps[i], 32, 64);
  }
  if (lane < 16) {
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][at + i] = ps[i];
  }
  if (li == 0 && held) atomicAdd(&cnt[a.experts], held);
  __syncthreads();
  for (int e = tid; e < a.experts; e += kRouteThreads)
    a.psum[(int64_t)blockIdx.x * a.experts + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
  for (int e = tid; e <= a.experts; e += kRouteThreads) a.hist[(int64_t)blockIdx.x * (a.experts + 1) + e] = cnt[e];
}

// Counts, slope and loss from the workgroups' sums, by one workgroup: as many
// threads per expert as there are.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void route_sum_kernel(RouteArgs a) {
  __shared__ int n_tokens;
  __shared__ int c_part[kSumThreads];
  __shared__ double p_part[kSumThreads];
  const int tid = threadIdx.x;
  const int wide = a.experts > 1 ? 1 << (32 - __clz(a.experts - 1)) : 1;  // experts, up to a power of two
  const int groups = kSumThreads / wide, e = tid & (wide - 1);
  int c = 0, n = 0;
  double p = 0.0;
  if (e < a.experts)
    for (int b = tid / wide; b < a.blocks; b += groups) {
      c += a.hist[(int64_t)b * (a.experts + 1) + e];
      p += a.psum[(int64_t)b * a.experts + e];
    }
  if (tid < 64) {
    for (int b = tid; b < a.blocks; b += 64) n += a.hist[(int64_t)b * (a.experts + 1) + a.experts];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) n += __shfl_xor(n, off, 64);
    if (tid == 0) n_tokens = n;
  }
  c_part[tid] = c;
  p_part[tid] = p;
  __syncthreads();
  double loss = 0.0;
  if (tid < a.experts) {
    for (int g = 1; g < groups; ++g) {
      c += c_part[g * wide + tid];
      p += p_part[g * wide + tid];
    }
    const double t = n_tokens;
    const float slope = n_tokens ? (float)c * (float)((double)a.experts / (t * t * (double)a.topk)) : 0.0f;
    a.counts[tid] = c;
    a.slope[tid] = slope;
    loss = (double)slope * p;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) loss += __shfl_xor(loss, off, 64);
  __syncthreads();
  if ((tid & 63) == 0) p_part[tid >> 6] = loss;
  __syncthreads();
  if (tid == 0) {
    double l = 0.0;
    for (int w = 0; w < kSumThreads / 64; ++w) l += p_part[w];
    *a.loss = (float)l;
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(RouteArgs a) {
  const int tid = threadIdx.x, li = tid & 15, lane = tid & 63, at = li * V;
  float slope[V];
#pragma unroll
  for (int i = 0; i < V; ++i) slope[i] = 0.0f;
  if (a.dloss) {
    const float d = *a.dloss;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at + i < a.experts) slope[i] = d * a.slope[at + i];
  }
  for (int64_t t0 = (int64_t)blockIdx.x * kRouteGroups; t0 < a.tokens; t0 += (int64_t)gridDim.x * kRouteGroups) {
    const int64_t t = t0 + (tid >> 4);
    const bool there = t < a.tokens;
    const bool real = there && (!a.mask || a.mask[t]);
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float v[V];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = -__builtin_inff();
    if (real) load_logits<T, V>(v, row, at, a.experts);
#pragma unroll
    for (int i = 0; i < V; ++i) top = umax32(top, key_of(v[i]));
    top = row16_max(top);
    const float most = logit_of(top);
    float s = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = top == 0 ? 0.0f : weight_of(v[i], most);
      s += v[i];
      dot += v[i] * slope[i];
    }
    s = row16_sum(s);
    dot = row16_sum(dot);
    const float inv = top == 0 ? 0.0f : 1.0f / s;
    dot *= inv;

    // the weights' part: an addition to the chosen experts' elements each, and
    // (where they are not normalized) one more dot product
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.0f;
    if (a.dweights) {
      float total = 0.0f, along = 0.0f;  // sums over the chosen of e^ and of e^ dw
      for (int j = li; j < a.topk; j += 16) {
        const int e = real ? a.expert[t * a.topk + j] : -1;
        if (e >= 0 && e < a.experts) {
          float l;
          if constexpr (sizeof(T) == 2) l = bf_lo(row[e]);
          else l = row[e];
          const float w = weight_of(l, most);
          total += w;
          along += w * a.dweights[t * a.topk + j];
        }
      }
      total = row16_sum(total);
      along = row16_sum(along);
      const float unit = top == 0 || (a.normalize && total == 0.0f) ? 0.0f : (a.normalize ? 1.0f / total : inv);
      along *= unit;
      if (!a.normalize) dot += along;
      for (int base = 0; base < a.topk; base += 16) {
        int e = -1;
        float add = 0.0f;
        if (real && base + li < a.topk) {
          e = a.expert[t * a.topk + base + li];
          if (e >= 0 && e < a.experts) {
            float l;
            if constexpr (sizeof(T) == 2) l = bf_lo(row[e]);
            else l = row[e];
            add = weight_of(l, most) * unit * (a.dweights[t * a.topk + base + li] - (a.normalize ? along : 0.0f));
          }
        }
        const int last = min(a.topk - base, 16);
        for (int j = 0; j < last; ++j) {
          const int ej = __shfl(e, (lane & 48) | j, 64);
          const float aj = __shfl(add, (lane & 48) | j, 64);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (at + i == ej) d[i] += aj;
        }
      }
    }
    if (there) {
      T* out = static_cast<T*>(a.dlogits) + t * a.ld_dlogits;
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = top == 0 ? 0.0f : d[i] + v[i] * inv * (slope[i] - dot);
      if constexpr (V >= 8) {
#pragma unroll
        for (int c = 0; c < V / 8; ++c) {
          Chunk<T> k;
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = d[8 * c + e];
          k.set(w);
          k.store(out + at + 8 * c, a.experts - at - 8 * c);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at + i < a.experts) {
            if constexpr (sizeof(T) == 2) out[at + i] = __builtin_bit_cast(uint16_t, (__bf16)d[i]);
            else out[at + i] = d[i];
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
  a.blocks = (int)route_blocks(p.tokens);
  a.psum = static_cast<float*>(p.workspace);
  a.hist = reinterpret_cast<int32_t*>(a.psum + a.blocks * p.experts);
  a.dweights = p.dweights;
  a.dloss = p.dloss;
  a.dlogits = p.dlogits;
  a.ld_dlogits = p.ld_dlogits;
  return a;
}

template <typename T, int V>
hipError_t route(const RouteArgs& a, bool given, hipStream_t st) {
  if (given) route_kernel<T, V, true><<<(unsigned)a.blocks, kRouteThreads, 0, st>>>(a);
  else route_kernel<T, V, false><<<(unsigned)a.blocks, kRouteThreads, 0, st>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  route_sum_kernel<<<1, kSumThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t route_back(const RouteArgs& a, hipStream_t st) {
  const int64_t groups = (a.tokens + kRouteGroups - 1) / kRouteGroups, most = 8 * (int64_t)cu_count(stream_device(st));
  route_backward_kernel<T, V><<<(unsigned)(groups < most ? groups : most), kRouteThreads, 0, st>>>(a);
  return hipGetLastError();
}

// experts per lane: as few powers of two as hold them
template <typename T, bool BACK>
hipError_t route_any(const RouteArgs& a, bool given, hipStream_t st) {
  auto go = [&](auto v) {
    if constexpr (BACK) return route_back<T, decltype(v)::value>(a, st);
    else return route<T, decltype(v)::value>(a, given, st);
  };
  if (a.experts <= 16) return go(std::integral_constant<int, 1>{});
  if (a.experts <= 32) return go(std::integral_constant<int, 2>{});
  if (a.experts <= 64) return go(std::integral_constant<int, 4>{});
  if (a.experts <= 128) return go(std::integral_constant<int, 8>{});
  if (a.experts <= 256) return go(std::integral_constant<int, 16>{});
  if (a.experts <= 512) return go(std::integral_constant<int, 32>{});
  return go(std::integral_constant<int, 64>{});
}

}  // namespace

// workgroups of the forward pass, each of which leaves its sums
int64_t route_blocks(int64_t tokens) {
  const int64_t n = (tokens + kRouteGroups * kRouteTokens - 1) / (kRouteGroups * kRouteTokens);
  return n < 1 ? 1 : (n < kRouteMaxBlocks ? n : kRouteMaxBlocks);
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
