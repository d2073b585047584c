// Routing of tokens to experts (include/pop_route.h): scores, bias, groups, the k best, weights.
//
// L lanes per token (1 to 32, a power of two) with V neighbouring experts each, so that among equal values the
// lowest lane, and in it the lowest place, is the lower expert. A choice value is kept as an unsigned key in
// the order of the floats (0: cannot be chosen). A lane sorts its keys in fours. k times: the largest of the
// lanes' first keys; the first lane that has it writes it down and moves up what stands behind it. At the end the
// chosen have a lane each, which finds the place of its key among all (they stand in shared memory) and computes the
// score, from the key or (with a bias) the logit again, so that the loop carries keys alone.
//
// UNIQUE: a bf16 logit fills half a key, and where the logits are the order (softmax without a bias) the other half
// holds the expert, from the top down. Then no two keys are equal and the largest key names its expert: there is no
// first lane and no place to find.
//
// What bounds it: few tokens, the k dependent steps (32 tokens, 256 experts in 8 groups, k = 8: 3.9 us; 8 experts,
// k = 2: 2.1); many, the instructions. 65,536 tokens, k = 6: 100 experts 11.6 us from bf16 (1.4 TB/s; 25 with keys of
// the other kind; 13.8 where the weights need the sum), 19.3 from float32 (1.5 TB/s); 64 experts 12.4. 256 experts in 8 groups, sigmoid and bias, k = 8: 4096
// tokens 7.0 us, 65,536 tokens 70 us. From 129 experts on a token has a whole warp, which finds its
// largest key in one instruction (16 lanes with 16 experts: 8.7 us for 4096 tokens); below that a warp has
// several tokens (a warp each: 65,536 x 100 from bf16 20.1 us instead of 11.6, float32 35 instead of 19, and less than 1 us
// gained for 64 tokens).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "pop_device.cuh"
#include "pop_qinternal.h"
#include "pop_route.h"

namespace pop {
namespace {

constexpr int RT_WARPS = 4;
struct RouteArgs {
  const void* logits;
  long long ld;
  const float* bias;
  int T, E, k, sigmoid, G, top_groups, group_sum, renorm;
  float scale;
  int* experts;
  float* weights;
  int* counts;
};

__device__ __forceinline__ float key_float(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// Key of a choice value; 0 for one that cannot be chosen (NaN, -infinity). + 0: -0 and +0 tie.
__device__ __forceinline__ uint32_t choice_key(float c) { return c >= -3.402823466e38f ? float_key(c + 0.f) : 0u; }

// What a logit counts as: -infinity where it is not live.
__device__ __forceinline__ float live_logit(float l) { return l == l ? fminf(l, 3.402823466e38f) : -INFINITY; }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, long long at) {
  if (BF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + at)) << 16);
  return __ldg(static_cast<const float*>(p) + at);
}

// A lane's V logits, n of which there are; the others are not live. VEC: four at a time.
template <bool BF16, int V, bool VEC>
__device__ __forceinline__ void load_logits(const void* p, long long at, int n, float (&l)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += VEC ? 4 : 1) {
    if (VEC) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < n) {
        if (BF16) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at + i));
          v = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
        } else {
          v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + i));
        }
      }
      l[i] = live_logit(v.x), l[i + 1] = live_logit(v.y), l[i + 2] = live_logit(v.z), l[i + 3] = live_logit(v.w);
    } else {
      l[i] = i < n ? live_logit(load_logit<BF16>(p, at + i)) : -INFINITY;
    }
  }
}

// The bias of a lane's experts.
template <int V, bool VEC>
__device__ __forceinline__ void load_bias(const float* p, int n, float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += VEC ? 4 : 1) {
    if (VEC) {
      const float4 v = i < n ? __ldg(reinterpret_cast<const float4*>(p + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
    } else {
      b[i] = i < n ? __ldg(p + i) : 0.f;
    }
  }
}

constexpr unsigned ALL = 0xffffffffu;

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(ALL, v);
  } else {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(ALL, v, o));
    return v;
  }
}
template <int V>
__device__ __forceinline__ uint32_t best_of(const uint32_t (&key)[V]) {
  uint32_t m = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = max(m, key[i]);
  return m;
}

// The two largest of (a1 >= a2) and (b1 >= b2).
__device__ __forceinline__ void merge2(uint32_t& a1, uint32_t& a2, uint32_t b1, uint32_t b2) {
  const uint32_t lo = min(a1, b1);
  a1 = max(a1, b1);
  a2 = max(lo, max(a2, b2));
}

// Larger first.
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t lo = min(a, b);
  a = max(a, b);
  b = lo;
}

// Unique keys: the logit's bits, in order, above 0xffff - expert. Smaller ones than this cannot be chosen (NaN
// counts as -infinity, and -infinity's bits become 0x007f).
constexpr uint32_t UNIQUE_LIVE = 0x00800000u;

__device__ __forceinline__ float unique_float(uint32_t key) {
  return fminf(key_float(key >= 0x80000000u ? key & 0xffff0000u : key | 0xffffu), 3.402823466e38f);
}

// The keys of a lane's V logits, of experts from e0 on, n of which there are; and the logits, two to a word, -infinity
// where they are not live.
template <int V, bool VEC>
__device__ __forceinline__ void unique_keys(const void* p, long long at, int e0, int n, uint32_t (&key)[V],
                                            uint32_t (&both)[V / 2]) {
  const uint16_t* l = static_cast<const uint16_t*>(p) + at;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    uint32_t* w = both + i / 2;
    w[0] = w[1] = 0xff80ff80u;  // -infinity
    if (VEC) {
      if (i < n) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(l + i));
        w[0] = u.x, w[1] = u.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) w[j / 2] = __byte_perm(w[j / 2], __ldg(l + i + j), j % 2 ? 0x5410 : 0x3254);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // NaN to -infinity, -0 to 0
      asm("max.bf16x2 %0, %0, %1;\n\tadd.rn.bf16x2 %0, %0, %2;" : "+r"(w[j]) : "r"(0xff80ff80u), "r"(0u));
      const uint32_t u = w[j] ^ 0x80008000u ^ ((w[j] >> 15 & 0x00010001u) * 0x7fffu);
      const uint32_t x = 0xffffu - static_cast<uint32_t>(e0 + i + 2 * j);
      key[i + 2 * j] = __byte_perm(u, x, 0x1054);
      key[i + 2 * j + 1] = __byte_perm(u, x - 1u, 0x3254);
    }
  }
}

template <bool BF16, bool UNIQUE, int L, int V, bool VEC>
__global__ void __launch_bounds__(32 * RT_WARPS) k_route(const __grid_constant__ RouteArgs a) {
  constexpr int TOK = 32 / L;  // tokens of a warp
  constexpr int K = L * V < POP_ROUTE_MAX_TOP_K ? L * V : POP_ROUTE_MAX_TOP_K;
  __shared__ uint32_t s_key[RT_WARPS][TOK][K];  // the chosen: keys, then scores
  __shared__ int s_e[RT_WARPS][TOK][K];         // lanes and which of equal keys, then experts
  __shared__ uint32_t s_all[RT_WARPS][V][32], s_grp[RT_WARPS][TOK][L * V];  // (all keys: place, lane)
  __shared__ int s_count[POP_ROUTE_MAX_EXPERTS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (L - 1), tok = lane / L;
  const int t0 = (blockIdx.x * RT_WARPS + warp) * TOK;
  const int t = min(t0 + tok, a.T - 1);  // (the last warp's spare lanes do the last token again)
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += 32 * RT_WARPS) s_count[e] = 0;
    __syncthreads();
  }
  const int e0 = sub * V;
  uint32_t key[V];
  float top = 0.f, sum = 1.f;
  if (UNIQUE) {
    uint32_t both[V / 2];
    unique_keys<V, VEC>(a.logits, t * a.ld + e0, e0, a.E - e0, key, both);
    if (!a.renorm) {  // (renormalised weights do not depend on the sum)
      top = unique_float(lanes_max<L>(best_of(key)));
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        sum += expf(fminf(i % 2 ? bf16hi(both[i / 2]) : bf16lo(both[i / 2]), 3.402823466e38f) - top);
      sum = lanes_sum<L>(sum);
    }
  } else {
    float l[V];
    load_logits<BF16, V, VEC>(a.logits, t * a.ld + e0, a.E - e0, l);
    float bias[V];
    if (a.bias) load_bias<V, VEC>(a.bias + e0, a.E - e0, bias);
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = 0u;
        if (l[i] != -INFINITY) {
          const float p = __frcp_rn(1.f + expf(-l[i]));
          key[i] = choice_key(a.bias ? p + bias[i] : p);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = choice_key(l[i]);
      const uint32_t m = lanes_max<L>(best_of(key));
      top = m ? key_float(m) : 0.f;
      if (a.bias || !a.renorm) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          l[i] = key[i] ? expf(l[i] - top) : 0.f;
          sum += l[i];
        }
        sum = lanes_sum<L>(sum);
      }
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i]) key[i] = choice_key(l[i] / sum + bias[i]);
      }
    }
  }
  if (a.G > 1) {
    const int per = a.E / a.G, lanes = per / V;
    if (lanes * V == per && (lanes & (lanes - 1)) == 0) {
      // a group is a power of two of whole lanes
      uint32_t k1 = max(key[0], key[1]), k2 = min(key[0], key[1]);
#pragma unroll
      for (int i = 2; i < V; i += 2) merge2(k1, k2, max(key[i], key[i + 1]), min(key[i], key[i + 1]));
      for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t b1 = __shfl_xor_sync(ALL, k1, o), b2 = __shfl_xor_sync(ALL, k2, o);
        merge2(k1, k2, b1, b2);
      }
      if (a.group_sum == 2 && k2) k1 = float_key(key_float(k1) + key_float(k2) + 0.f);
      const int g = e0 / per;
      int before = 0;
      for (int j = 0; j < a.G; ++j) {
        const uint32_t u = __shfl_sync(ALL, k1, j * lanes, L);
        before += (u > k1 || (u == k1 && j < g)) ? 1 : 0;
      }
      if (before >= a.top_groups) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0u;
      }
    } else {
      uint32_t(*sk)[32] = s_all[warp], *sg = s_grp[warp][tok];
      const int l0 = lane - sub;
#pragma unroll
      for (int i = 0; i < V; ++i) sk[i][lane] = key[i];
      __syncwarp();
      for (int g = sub; g < a.G; g += L) {
        uint32_t k1 = 0, k2 = 0;
        for (int e = g * per; e < (g + 1) * per; ++e) merge2(k1, k2, sk[e % V][l0 + e / V], 0u);
        if (a.group_sum == 2 && k2) k1 = float_key(key_float(k1) + key_float(k2) + 0.f);
        sg[g] = k1;
      }
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < V; ++i) {
        const int g = min(e0 + i, a.E - 1) / per;
        int before = 0;
        for (int j = 0; j < a.G; ++j) before += (sg[j] > sg[g] || (sg[j] == sg[g] && j < g)) ? 1 : 0;
        if (before >= a.top_groups) sk[i][lane] = 0u;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = sk[i][lane];
    }
  }
  if (!UNIQUE) {  // for the places of the chosen
#pragma unroll
    for (int i = 0; i < V; ++i) s_all[warp][i][lane] = key[i];
  }
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    order(key[i], key[i + 1]), order(key[i + 2], key[i + 3]);
    order(key[i], key[i + 2]), order(key[i + 1], key[i + 3]);
    order(key[i + 1], key[i + 2]);
  }
  uint32_t last = 0;
  int equal = 0;  // keys equal to the one a lane gave last that it had given before
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 4; i < V; i += 4) best = max(best, key[i]);
    const uint32_t m = lanes_max<L>(best);
    bool mine = UNIQUE;
    if (!UNIQUE) {
      unsigned has = __ballot_sync(ALL, best == m);
      if (L < 32) has &= ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
      mine = lane == __ffs(has) - 1;
    }
    if (UNIQUE ? sub == 0 : mine) s_key[warp][tok][j] = m;
    if (!UNIQUE && mine) {
      equal = m == last ? equal + 1 : 0;
      last = m;
      s_e[warp][tok][j] = lane | equal << 8;
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (mine && key[i] == m) {
        key[i] = key[i + 1], key[i + 1] = key[i + 2], key[i + 2] = key[i + 3], key[i + 3] = 0u;
        if (!UNIQUE) mine = false;
      }
    }
  }
  __syncwarp();
  // the chosen, a lane each: scores, then weights
  const bool live = t0 + tok < a.T;
  if (UNIQUE) top = unique_float(s_key[warp][tok][0]);
  __syncwarp();  // (the first one's key becomes a score)
  float total = 0.f;
  for (int j = sub; j < a.k; j += L) {
    const uint32_t m = s_key[warp][tok][j];
    float w = 0.f;
    if (UNIQUE) {
      if (m >= UNIQUE_LIVE) w = expf(unique_float(m) - top) / sum;
      s_e[warp][tok][j] = m >= UNIQUE_LIVE ? static_cast<int>(0xffffu - (m & 0xffffu)) : -1;
    } else {
      int e = -1;
      if (m) {
        const int from = s_e[warp][tok][j];
        unsigned hits = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) hits |= s_all[warp][i][from & 31] == m ? 1u << i : 0u;
        for (int i = from >> 8; i; --i) hits &= hits - 1;
        e = (from & (L - 1)) * V + __ffs(hits) - 1;
        float v = key_float(m);
        if (a.bias) v = live_logit(load_logit<BF16>(a.logits, t * a.ld + e));
        if (!a.sigmoid)
          w = expf(v - top) / sum;
        else
          w = a.bias ? __frcp_rn(1.f + expf(-v)) : v;
      }
      s_e[warp][tok][j] = e;
    }
    s_key[warp][tok][j] = __float_as_uint(w);
    total += w;
  }
  total = lanes_sum<L>(total);
  for (int j = sub; j < a.k && live; j += L) {
    const int e = s_e[warp][tok][j];
    float w = __uint_as_float(s_key[warp][tok][j]);
    if (a.renorm) w = total > 0.f ? w / total : 0.f;
    const size_t at = static_cast<size_t>(t) * a.k + j;
    a.experts[at] = e;
    a.weights[at] = w * a.scale;
    if (a.counts && e >= 0) atomicAdd(&s_count[e], 1);
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 32 * RT_WARPS)
      if (s_count[e]) atomicAdd(a.counts + e, s_count[e]);
  }
}

template <bool BF16, bool UNIQUE, int L, int V>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
  const int grid = (a.T + 32 / L * RT_WARPS - 1) / (32 / L * RT_WARPS);
  // four values a load where rows and runs of four start on such a boundary and end with the experts
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (BF16 ? 8 : 16) == 0 &&
                   reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  return launch_plain(vec ? k_route<BF16, UNIQUE, L, V, true> : k_route<BF16, UNIQUE, L, V, false>, dim3(grid), 32 * RT_WARPS, st, a);
}

template <bool BF16, bool UNIQUE>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
  if (a.E <= 8) return launch_route<BF16, UNIQUE, 1, 8>(a, st);
  if (a.E <= 16) return launch_route<BF16, UNIQUE, 1, 16>(a, st);
  if (a.E <= 32) return launch_route<BF16, UNIQUE, 2, 16>(a, st);
  if (a.E <= 64) return launch_route<BF16, UNIQUE, 4, 16>(a, st);
  if (a.E <= 128) return launch_route<BF16, UNIQUE, 8, 16>(a, st);
  return launch_route<BF16, UNIQUE, 32, 8>(a, st);
}

thread_local std::string g_route_msg;

pop_status route_fail(pop_status s, const char* msg) {
  if (s == POP_ERR_CUDA) cudaGetLastError();  // it is reported here: a later call is not to find it
  try {
    g_route_msg = msg;
  } catch (...) {
  }
  return s;
}

}  // namespace
}  // namespace pop

extern "C" {

const char* pop_route_last_error(void) { return pop::g_route_msg.c_str(); }

pop_status pop_route(const pop_route_config* cfg, const void* logits, int logits_bf16, long long ld_logits,
                     const float* bias, int T, int* experts, float* weights, int* counts, void* stream) {
  using namespace pop;
  const auto bad = [](const char* m) { return route_fail(POP_ERR_INVALID_ARG, m); };
  if (!cfg) return bad("pop_route: cfg is NULL");
  const pop_route_config& c = *cfg;
  if (c.n_experts < 1 || c.n_experts > POP_ROUTE_MAX_EXPERTS) return bad("pop_route: n_experts out of range");
  if (c.score != POP_ROUTE_SOFTMAX && c.score != POP_ROUTE_SIGMOID) return bad("pop_route: unknown score");
  if (c.n_groups < 1 || c.n_experts % c.n_groups) return bad("pop_route: n_groups must divide n_experts");
  if (c.top_groups < 1 || c.top_groups > c.n_groups) return bad("pop_route: top_groups outside [1, n_groups]");
  if (c.top_k < 1 || c.top_k > POP_ROUTE_MAX_TOP_K || c.top_k > c.top_groups * (c.n_experts / c.n_groups))
    return bad("pop_route: top_k outside [1, min(POP_ROUTE_MAX_TOP_K, experts of top_groups groups)]");
  if (c.group_sum != 1 && c.group_sum != 2) return bad("pop_route: group_sum must be 1 or 2");
  if (c.group_sum == 2 && c.score == POP_ROUTE_SOFTMAX && !bias)
    return bad("pop_route: group_sum 2 needs sigmoid scores or a bias");
  if ((c.renorm != 0 && c.renorm != 1) || !std::isfinite(c.scale))
    return bad("pop_route: renorm must be 0 or 1, scale finite");
  if (logits_bf16 != 0 && logits_bf16 != 1) return bad("pop_route: logits_bf16 must be 0 or 1");
  if (T < 0 || T > (1 << 27)) return bad("pop_route: T outside [0, 2^27]");
  const auto off = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
  if (T == 0 && !counts) return POP_OK;
  if (T > 0) {
    if (!logits || !experts || !weights) return bad("pop_route: NULL logits, experts or weights");
    if (ld_logits < c.n_experts) return bad("pop_route: ld_logits < n_experts");
    if (off(logits, logits_bf16 ? 2 : 4) || off(bias, 4) || off(experts, 4) || off(weights, 4))
      return bad("pop_route: a pointer is not aligned to its element");
  }
  if (off(counts, 4)) return bad("pop_route: counts is not aligned to its element");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return route_fail(dev, "pop_route: needs an sm_103 device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (counts) e = cudaMemsetAsync(counts, 0, sizeof(int) * c.n_experts, st);
  if (e != cudaSuccess) return route_fail(POP_ERR_CUDA, cudaGetErrorString(e));
  if (T == 0) return POP_OK;  // no slots: the counts are 0
  RouteArgs a{logits,       ld_logits,   bias,     T,       c.n_experts, c.top_k, c.score == POP_ROUTE_SIGMOID,
              c.n_groups,   c.top_groups, c.group_sum, c.renorm, c.scale,     experts, weights,
              counts};
  if (!logits_bf16)
    e = launch_route<false, false>(a, st);
  else if (a.sigmoid || a.bias)
    e = launch_route<true, false>(a, st);
  else
    e = launch_route<true, true>(a, st);
  return e == cudaSuccess ? POP_OK : route_fail(POP_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
