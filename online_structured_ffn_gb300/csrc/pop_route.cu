// Routing of tokens to experts (include/pop_route.h): scores, bias, groups, the k best, weights.
//
// One warp per token; lane j holds experts j, j + 32, ... A choice value is kept as an unsigned key in
// the order of the floats (0: not live), so that the best is a warp maximum and a tie's lower index a
// warp minimum.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "pop_device.cuh"
#include "pop_qinternal.h"
#include "pop_route.h"

namespace pop {
namespace {

constexpr int RT_WARPS = 8;
constexpr int RT_VALS = POP_ROUTE_MAX_EXPERTS / 32;

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

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, long long i) {
  if (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  return static_cast<const float*>(p)[i];
}

template <bool BF16>
__global__ void __launch_bounds__(32 * RT_WARPS) k_route(RouteArgs a) {
  __shared__ uint32_t s_key[RT_WARPS][POP_ROUTE_MAX_EXPERTS];
  __shared__ uint32_t s_grp[RT_WARPS][POP_ROUTE_MAX_EXPERTS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * RT_WARPS + warp;
  if (t >= a.T) return;
  constexpr unsigned ALL = 0xffffffffu;
  float s[RT_VALS];
  uint32_t key[RT_VALS];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < RT_VALS; ++i) {
    const int e = lane + 32 * i;
    float l = -INFINITY;
    if (e < a.E) l = load_logit<BF16>(a.logits, t * a.ld + e);
    l = l == l ? fminf(l, 3.402823466e38f) : -INFINITY;
    s[i] = l;
    top = fmaxf(top, l);
  }
  float sum = 0.f;
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, o));
  }
#pragma unroll
  for (int i = 0; i < RT_VALS; ++i) {
    const int e = lane + 32 * i;
    const float l = s[i];
    const bool live = l != -INFINITY;
    key[i] = choice_key(l);
    s[i] = 0.f;
    if (live) s[i] = a.sigmoid ? 1.f / (1.f + expf(-l)) : expf(l - top);
    sum += s[i];
    if (a.sigmoid && live) key[i] = choice_key(a.bias ? s[i] + a.bias[e] : s[i]);
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i) {
      s[i] = key[i] ? s[i] / sum : 0.f;
      if (a.bias && key[i]) key[i] = choice_key(s[i] + a.bias[lane + 32 * i]);
    }
  }
  if (a.G > 1) {
    const int per = a.E / a.G;
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i)
      if (lane + 32 * i < a.E) s_key[warp][lane + 32 * i] = key[i];
    __syncwarp();
    for (int g = lane; g < a.G; g += 32) {
      uint32_t k1 = 0, k2 = 0;
      for (int j = 0; j < per; ++j) {
        const uint32_t v = s_key[warp][g * per + j];
        if (v > k1) {
          k2 = k1;
          k1 = v;
        } else if (v > k2) {
          k2 = v;
        }
      }
      if (a.group_sum == 2 && k2) k1 = float_key(key_float(k1) + key_float(k2) + 0.f);
      s_grp[warp][g] = k1;
    }
    __syncwarp();
    // rank of every group among the others: a group stays if fewer than top_groups come before it
    uint32_t stay[RT_VALS];
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i) {
      const int g = lane + 32 * i;
      stay[i] = 0;
      if (g < a.G) {
        const uint32_t v = s_grp[warp][g];
        int before = 0;
        for (int j = 0; j < a.G; ++j) {
          const uint32_t u = s_grp[warp][j];
          before += (u > v || (u == v && j < g)) ? 1 : 0;
        }
        stay[i] = before < a.top_groups ? 1u : 0u;
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i)
      if (lane + 32 * i < a.G) s_grp[warp][lane + 32 * i] = stay[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i)
      if (lane + 32 * i < a.E && !s_grp[warp][(lane + 32 * i) / per]) key[i] = 0u;
  }
  int my_e = -1;      // slot `lane` of the token
  float my_w = 0.f;
  float total = 0.f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(ALL, best);
    if (best == 0) break;
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int i = RT_VALS - 1; i >= 0; --i)
      if (key[i] == best) at = lane + 32 * i;
    at = __reduce_min_sync(ALL, at);
    float w = 0.f;
#pragma unroll
    for (int i = 0; i < RT_VALS; ++i)
      if (static_cast<unsigned>(lane + 32 * i) == at) {
        w = s[i];
        key[i] = 0u;
      }
    w = __shfl_sync(ALL, w, at & 31u);
    total += w;
    if (lane == j) {
      my_e = static_cast<int>(at);
      my_w = w;
    }
  }
  if (a.renorm) my_w = total > 0.f ? my_w / total : 0.f;
  if (lane < a.k) {
    const size_t o = static_cast<size_t>(t) * a.k + lane;
    a.experts[o] = my_e;
    a.weights[o] = my_w * a.scale;
    if (a.counts && my_e >= 0) atomicAdd(a.counts + my_e, 1);
  }
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
  const int grid = (T + RT_WARPS - 1) / RT_WARPS;
  if (logits_bf16)
    k_route<true><<<grid, 32 * RT_WARPS, 0, st>>>(a);
  else
    k_route<false><<<grid, 32 * RT_WARPS, 0, st>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? POP_OK : route_fail(POP_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
