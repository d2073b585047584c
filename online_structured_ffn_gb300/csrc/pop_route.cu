// Routing of tokens to experts (include/pop_route.h): scores, bias, groups, the k best, weights.
//
// L lanes per token (1 to 16, a power of two) with V = 8 or 16 neighbouring experts each, so that among equal
// values the lowest lane, and in it the lowest place, is the lower expert. A choice value is kept as an
// unsigned key in the order of the floats (0: cannot be chosen). k times: the largest of the lanes' best keys, the
// first lane that has it, which writes it down and looks for its next best. The chosen scores are computed
// at the end, from the keys or (with a bias) the logits again, a lane each, so that the loop carries keys alone.
// What bounds it is the instructions: some 200 a token for 100 experts and k = 6.
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

constexpr unsigned ALL = 0xffffffffu;

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(ALL, v, o));
  return v;
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

template <bool BF16, int L, int V, bool VEC>
__global__ void __launch_bounds__(32 * RT_WARPS) k_route(const __grid_constant__ RouteArgs a) {
  constexpr int TOK = 32 / L;  // tokens of a warp
  __shared__ uint32_t s_key[RT_WARPS][TOK][POP_ROUTE_MAX_TOP_K];  // the chosen: keys, then scores
  __shared__ int s_e[RT_WARPS][TOK][POP_ROUTE_MAX_TOP_K];
  __shared__ float s_top[RT_WARPS][TOK], s_sum[RT_WARPS][TOK];
  __shared__ uint32_t s_all[RT_WARPS][TOK][L * V], s_grp[RT_WARPS][TOK][L * V];
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
  {
    float l[V];
    load_logits<BF16, V, VEC>(a.logits, t * a.ld + e0, a.E - e0, l);
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        key[i] = 0u;
        if (l[i] != -INFINITY) {
          const float p = __frcp_rn(1.f + expf(-l[i]));
          key[i] = choice_key(a.bias ? p + __ldg(a.bias + e0 + i) : p);
        }
      }
    } else {
      top = l[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = lanes_max<L>(top);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = choice_key(l[i]);
      if (a.bias || !a.renorm) {  // (renormalised weights do not depend on the sum)
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
          if (key[i]) key[i] = choice_key(l[i] / sum + __ldg(a.bias + e0 + i));
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
      uint32_t *sk = s_all[warp][tok], *sg = s_grp[warp][tok];
#pragma unroll
      for (int i = 0; i < V; ++i) sk[e0 + i] = key[i];
      __syncwarp();
      for (int g = sub; g < a.G; g += L) {
        uint32_t k1 = 0, k2 = 0;
        for (int j = 0; j < per; ++j) merge2(k1, k2, sk[g * per + j], 0u);
        if (a.group_sum == 2 && k2) k1 = float_key(key_float(k1) + key_float(k2) + 0.f);
        sg[g] = k1;
      }
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < V; ++i) {
        const int g = min(e0 + i, a.E - 1) / per;
        int before = 0;
        for (int j = 0; j < a.G; ++j) before += (sg[j] > sg[g] || (sg[j] == sg[g] && j < g)) ? 1 : 0;
        if (before >= a.top_groups) sk[e0 + i] = 0u;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = sk[e0 + i];
    }
  }
  uint32_t best = best_of(key);
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    const uint32_t m = lanes_max<L>(best);
    unsigned has = __ballot_sync(ALL, best == m);
    if (L < 32) has &= ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
    if (lane == __ffs(has) - 1) {
      unsigned hits = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] == m) hits |= 1u << i, key[i] = 0u;
      const int at = __ffs(hits) - 1;
      hits &= hits - 1;
      if (hits && m) {  // a tie within the lane: the others stay
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (hits >> i & 1u) key[i] = m;
      }
      best = best_of(key);
      s_key[warp][tok][j] = m;
      s_e[warp][tok][j] = m ? e0 + at : -1;
    }
  }
  if (sub == 0) s_top[warp][tok] = top, s_sum[warp][tok] = sum;
  __syncwarp();
  // the scores of the chosen, a lane each
  const int n = min(TOK, a.T - t0) * a.k;
  for (int o = lane; o < n; o += 32) {
    const int u = o / a.k, j = o - u * a.k;
    const uint32_t m = s_key[warp][u][j];
    float w = 0.f;
    if (m) {
      float v = key_float(m);
      if (a.bias) v = live_logit(load_logit<BF16>(a.logits, (t0 + u) * a.ld + s_e[warp][u][j]));
      if (!a.sigmoid)
        w = expf(v - s_top[warp][u]) / s_sum[warp][u];
      else
        w = a.bias ? __frcp_rn(1.f + expf(-v)) : v;
    }
    s_key[warp][u][j] = __float_as_uint(w);
  }
  __syncwarp();
  const size_t out = static_cast<size_t>(t0) * a.k;
  for (int o = lane; o < n; o += 32) {
    const int u = o / a.k, j = o - u * a.k;
    const int e = s_e[warp][u][j];
    float w = __uint_as_float(s_key[warp][u][j]);
    if (a.renorm) {
      float total = 0.f;
      for (int i = 0; i < a.k; ++i) total += __uint_as_float(s_key[warp][u][i]);
      w = total > 0.f ? w / total : 0.f;
    }
    a.experts[out + o] = e;
    a.weights[out + o] = w * a.scale;
    if (a.counts && e >= 0) atomicAdd(&s_count[e], 1);
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 32 * RT_WARPS)
      if (s_count[e]) atomicAdd(a.counts + e, s_count[e]);
  }
}

template <bool BF16, int L, int V>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
  const int grid = (a.T + 32 / L * RT_WARPS - 1) / (32 / L * RT_WARPS);
  // four logits a load where rows and runs of four start on such a boundary and end with the experts
  const bool vec = a.E % 4 == 0 && a.ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % (BF16 ? 8 : 16) == 0;
  if (vec)
    k_route<BF16, L, V, true><<<grid, 32 * RT_WARPS, 0, st>>>(a);
  else
    k_route<BF16, L, V, false><<<grid, 32 * RT_WARPS, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
  if (a.E <= 8) return launch_route<BF16, 1, 8>(a, st);
  if (a.E <= 16) return launch_route<BF16, 1, 16>(a, st);
  if (a.E <= 32) return launch_route<BF16, 2, 16>(a, st);
  if (a.E <= 64) return launch_route<BF16, 4, 16>(a, st);
  if (a.E <= 128) return launch_route<BF16, 8, 16>(a, st);
  return launch_route<BF16, 16, 16>(a, st);
}

thread_local std::string g_route_msg;

pop_status route_fail(pop_status s, const char* msg) {
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
  if (T == 0) return POP_OK;
  if (!logits || !experts || !weights) return bad("pop_route: NULL logits, experts or weights");
  if (ld_logits < c.n_experts) return bad("pop_route: ld_logits < n_experts");
  const auto off = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
  if (off(logits, logits_bf16 ? 2 : 4) || off(bias, 4) || off(experts, 4) || off(weights, 4) || off(counts, 4))
    return bad("pop_route: a pointer is not aligned to its element");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return route_fail(dev, "pop_route: needs an sm_103 device");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (counts) e = cudaMemsetAsync(counts, 0, sizeof(int) * c.n_experts, st);
  if (e != cudaSuccess) return route_fail(POP_ERR_CUDA, cudaGetErrorString(e));
  RouteArgs a{logits,       ld_logits,   bias,     T,       c.n_experts, c.top_k, c.score == POP_ROUTE_SIGMOID,
              c.n_groups,   c.top_groups, c.group_sum, c.renorm, c.scale,     experts, weights,
              counts};
  e = logits_bf16 ? launch_route<true>(a, st) : launch_route<false>(a, st);
  return e == cudaSuccess ? POP_OK : route_fail(POP_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
