// Rows and matrices in e4m3 with a scale per block of 128: quantising, operand images, the grouping of
// tokens by expert and the weighted sum of the experts' outputs (include/pop_quant.h, pop_qinternal.h).
#include "pop_qdevice.cuh"

namespace pop {
namespace {

__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
}

// 32 bytes, aligned to 32, in one load: a lane's values are whole sectors, which two loads of 16 bytes each fetched twice.
__device__ __forceinline__ void ldg_sector(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}

// The places of a CTA's own pairs, [p0, p0 + n) of all, found from the experts of all of them: how many pairs of the
// same expert come before, and where the expert's rows begin. row[i] is that of pair p0 + i.
struct Places {
  int total[POP_QMOE_MAX_EXPERTS], before[POP_QMOE_MAX_EXPERTS];
  int own[32 * POP_QMOE_MAX_TOP_K], row[32 * POP_QMOE_MAX_TOP_K];

  __device__ __forceinline__ void find(const QRowsOut& out, int pairs, int p0, int n, bool report) {
    for (int e = threadIdx.x; e < out.E; e += 256) total[e] = before[e] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < pairs; c += 8 * 256) {
      int es[8];  // eight loads on their way
#pragma unroll
      for (int i = 0; i < 8; ++i) es[i] = c + 256 * i < pairs ? __ldg(out.experts + c + 256 * i) : -1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int p = c + 256 * i, e = es[i];
        const bool is = static_cast<unsigned>(e) < static_cast<unsigned>(out.E);
        if (is) atomicAdd(&total[e], 1);
        if (is && p < p0) atomicAdd(&before[e], 1);
        if (p >= p0 && p < p0 + n) own[p - p0] = is ? e : -1;
        if (report && !is && e != -1) atomicOr(out.err, QERR_EXPERT);
      }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      int base = 0;
      for (int e0 = 0; e0 < out.E; e0 += 32) {
        const int e = e0 + static_cast<int>(threadIdx.x);
        const int rows = e < out.E ? qceil(total[e], out.G) * out.G : 0;
        int s = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if (static_cast<int>(threadIdx.x) >= o) s += v;
        }
        if (e < out.E) before[e] += base + s - rows;
        base += __shfl_sync(0xffffffffu, s, 31);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += 256) {
      const int e = own[i];
      int r = -1;
      if (e >= 0) {
        r = before[e];
        for (int j = 0; j < i; ++j) r += own[j] == e ? 1 : 0;
      }
      row[i] = r;
    }
    __syncthreads();
  }
};

// Eight lanes per block of 128, 16 values each. A CTA has 32 blocks: of one row (the blockIdx.y-th 32), or of the
// `per` whole rows that they hold. Bound by memory and nearly so by its instructions, of which every one counts:
// 16 values take two each for the quotient (packed; four, and 9.8 us, without), half a rounding, one for bf16's
// unpacking. 4096 x 4096 of bf16: 8.9 us (5.7 TB/s read and written), 16,384 x 4096 33.8 (6.0); 1001 x 11008 of float32
// 8.5 (6.6; 9.4 with loads of 16 bytes). Where the blocks do not fill a CTA's 32 groups the others idle: 16,384 x 4096 values in
// rows of 4096 6.0 TB/s, of 7168 (28 of 32) 5.8, 6144 5.4, 2880 5.2, 5120 (20 of 32) 4.8, 4608 4.4, 4224 (33 of 64) 4.0.
template <int KIND>
__global__ void __launch_bounds__(256) k_quantize_rows(const __grid_constant__ QRowsArgs in, const __grid_constant__ QRowsOut out, int per) {
  // Behind the kernel that places the rows (row_of) x is complete, as that one has waited for it: only the places, and
  // what an earlier call's kernels may still read, are then waited for, after the arithmetic.
  if (!out.row_of) {
    pdl_wait();
    pdl_trigger();
  }
  const int KB = qceil(in.K, QB);
  const int lane8 = threadIdx.x & 7, u = threadIdx.x >> 3;
  int row = blockIdx.x, kb = u + 32 * blockIdx.y;
  bool on = kb < KB;
  if (per > 1) {
    const int row_in = u / KB;
    row = blockIdx.x * per + row_in;
    kb = u - row_in * KB;
    on = row_in < per && row < in.M;
  }
  const int k0 = kb * QB + lane8 * 16;
  const int n8 = on ? min(max((in.K - k0) >> 3, 0), 2) : 0;  // runs of 8 values this lane has
  // The values, as they stand in memory: on their way while the places are looked for.
  uint4 raw[KIND == 1 ? 4 : 2];
#pragma unroll
  for (int i = 0; i < (KIND == 1 ? 4 : 2); ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
  float s = 0.f;
  if (KIND == 2) {
    const uint8_t* p = static_cast<const uint8_t*>(in.x) + static_cast<size_t>(row) * in.ldx + k0;
    if (n8 > 0) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      raw[0].x = a.x, raw[0].y = a.y;
    }
    if (n8 > 1) {
      const uint2 b = *reinterpret_cast<const uint2*>(p + 8);
      raw[0].z = b.x, raw[0].w = b.y;
    }
    if (on) s = in.xs[static_cast<size_t>(row) * in.lds + kb];
  } else {
    constexpr int SIZE = KIND == 0 ? 2 : 4, N16 = SIZE / 2;  // 16-byte loads of eight values
    const uint8_t* p = static_cast<const uint8_t*>(in.x) + (static_cast<size_t>(row) * in.ldx + k0) * SIZE;
    if (n8 > 1 && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N16; ++i) ldg_sector(p + 32 * i, raw[2 * i], raw[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < N16; ++j)
          if (n8 > i) raw[i * N16 + j] = ldg_stream(p + (i * N16 + j) * 16);
    }
  }
  __shared__ Places places;
  if (out.experts) {
    const int t0 = blockIdx.x * per, n = min(per, in.M - t0) * out.k;
    places.find(out, in.M * out.k, t0 * out.k, n, blockIdx.x == 0 && blockIdx.y == 0);
    if (blockIdx.y == 0)
      for (int i = threadIdx.x; i < n; i += 256) out.places[t0 * out.k + i] = places.row[i];
  }
  uint4 q = raw[0];
  if (KIND != 2) {
    float v[16];
    if (KIND == 0) {
      unpack8(raw[0], v);
      unpack8(raw[1], v + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const uint4 w = raw[KIND == 1 ? i / 4 : 0];
        v[i] = __uint_as_float(w.x), v[i + 1] = __uint_as_float(w.y), v[i + 2] = __uint_as_float(w.z), v[i + 3] = __uint_as_float(w.w);
      }
    }
    float a = __uint_as_float(AMAX_MIN_BITS);
#pragma unroll
    for (int i = 0; i < 16; i += 2) a = max_abs(a, v[i], v[i + 1]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a = max_abs(a, __shfl_xor_sync(0xffffffffu, a, o), 0.f);
    q = e4m3x16(v, BlockRatio(a));
    s = block_scale(a);
  }
  if (out.row_of) {
    pdl_wait();
    pdl_trigger();
  }
  if (!on) return;
  if (out.G == 0) {
    uint8_t* p = out.q + static_cast<size_t>(row) * out.ldq + k0;
    if (n8 > 1 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      *reinterpret_cast<uint4*>(p) = q;
    } else {
      if (n8 > 0) *reinterpret_cast<uint2*>(p) = make_uint2(q.x, q.y);
      if (n8 > 1) *reinterpret_cast<uint2*>(p + 8) = make_uint2(q.z, q.w);
    }
    if (lane8 == 0) out.s[static_cast<size_t>(row) * KB + kb] = s;
    return;
  }
  const int log_g = 31 - __clz(out.G);
  for (int j = 0; j < out.k; ++j) {
    const int r = out.experts  ? places.row[(row - blockIdx.x * per) * out.k + j]
                  : out.row_of ? __ldcg(out.row_of + static_cast<size_t>(row) * out.k + j)
                               : row;
    if (r < 0) continue;
    const int in_run = r & (out.G - 1);
    const size_t block = static_cast<size_t>(r >> log_g) * KB + kb;
    *reinterpret_cast<uint4*>(out.q + ((block * QB) << log_g) + image_at(in_run, lane8 * 16)) = q;
    if (lane8 == 0) out.s[(block << log_g) + in_run] = s;
  }
}

// One CTA per 128 x 128 block; thread (r, c) holds the 16-byte chunks c of rows r, r + 32, ...
__global__ void __launch_bounds__(256) k_pack_matrix(const void* __restrict__ W, const float* __restrict__ Ws, int N,
                                                     int K, uint8_t* __restrict__ img, float* __restrict__ sc,
                                                     int step, int part) {
  __shared__ uint32_t s_max;
  const int KB = qceil(K, QB);
  const int t = blockIdx.y, b = blockIdx.x;
  const size_t slot = (static_cast<size_t>(t) * KB + b) * step + part;
  float* scale = sc + static_cast<size_t>(t) * scale_stride(KB, step) + b * step + part;
  const int c = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int k0 = b * QB + c * 16;
  const int n8 = min(max((K - k0) >> 3, 0), 2);
  uint4* dst = reinterpret_cast<uint4*>(img + slot * QTILE);
  if (Ws) {
    for (int r = r0; r < QB; r += 32) {
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (t * QB + r < N) {
        const uint8_t* p = static_cast<const uint8_t*>(W) + static_cast<size_t>(t * QB + r) * K + k0;
        if (n8 > 0) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          q.x = v.x, q.y = v.y;
        }
        if (n8 > 1) {
          const uint2 v = *reinterpret_cast<const uint2*>(p + 8);
          q.z = v.x, q.w = v.y;
        }
      }
      dst[image_at(r, c * 16) >> 4] = q;
    }
    if (threadIdx.x == 0) *scale = Ws[static_cast<size_t>(t) * KB + b];
    return;
  }
  if (threadIdx.x == 0) s_max = AMAX_MIN_BITS;
  __syncthreads();
  float v[4][16];
  uint32_t m = AMAX_MIN_BITS;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 32 * i;
#pragma unroll
    for (int j = 0; j < 16; ++j) v[i][j] = 0.f;
    if (t * QB + r < N) {
      const uint8_t* p = static_cast<const uint8_t*>(W) + (static_cast<size_t>(t * QB + r) * K + k0) * 2;
      if (n8 > 0) unpack8(ldg_stream(p), v[i]);
      if (n8 > 1) unpack8(ldg_stream(p + 16), v[i] + 8);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[i][j]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_max, m);
  __syncthreads();
  const float a = __uint_as_float(s_max);
  const BlockRatio ratio(a);
#pragma unroll
  for (int i = 0; i < 4; ++i) dst[image_at(r0 + 32 * i, c * 16) >> 4] = e4m3x16(v[i], ratio);
  if (threadIdx.x == 0) *scale = block_scale(a);
}

// One CTA; warp w has the w-th part of the pairs. First every warp counts its pairs of each expert (lanes with the
// same expert find each other with a match), then the counts become first places (over the warps, and over the
// experts in whole runs), then every warp goes through its pairs again and numbers them, in ascending order. Bound by
// its dependent steps: 8192 pairs of 8 experts 10.6 us, beside products of 1200.
constexpr int PLAN_WARPS = 32;
__global__ void __launch_bounds__(32 * PLAN_WARPS) k_plan(const int* __restrict__ experts, int pairs, int E, int G,
                                                          int* __restrict__ counts, int* __restrict__ row_of,
                                                          unsigned* __restrict__ err) {
  __shared__ int s_at[PLAN_WARPS][POP_QMOE_MAX_EXPERTS];
  __shared__ int s_base[POP_QMOE_MAX_EXPERTS / 32];
  constexpr unsigned ALL = 0xffffffffu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < PLAN_WARPS * POP_QMOE_MAX_EXPERTS / 4; i += blockDim.x)
    reinterpret_cast<int4*>(&s_at[0][0])[i] = make_int4(0, 0, 0, 0);
  pdl_wait();  // the routing, and an earlier call's use of what is written here
  pdl_trigger();
  const int part = qceil(qceil(pairs, PLAN_WARPS), 32) * 32;
  const int p0 = min(pairs, warp * part), p1 = min(pairs, p0 + part);
  // 128 pairs at a time: the experts of four of them per lane, -1 for none
  int e[4];
  auto load = [&](int c, bool report) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = c + 32 * i + lane < p1 ? __ldg(experts + c + 32 * i + lane) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool is = static_cast<unsigned>(e[i]) < static_cast<unsigned>(E);
      if (report && !is && e[i] != -1) atomicOr(err, QERR_EXPERT);
      if (!is) e[i] = -1;
    }
  };
  if (p0 < p1) load(p0, true);
  __syncthreads();
  for (int c = p0; c < p1; c += 128) {
    if (c > p0) load(c, true);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + 32 * i >= p1) break;
      const unsigned same = __match_any_sync(ALL, e[i]);
      if (e[i] >= 0 && lane == __ffs(same) - 1) s_at[warp][e[i]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  int own = 0, before = 0;
  if (threadIdx.x < POP_QMOE_MAX_EXPERTS) {
    const int x = threadIdx.x;
    int at[PLAN_WARPS];
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) at[w] = s_at[w][x];
    int n = 0;
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) {
      s_at[w][x] = n;
      n += at[w];
    }
    if (x < E) counts[x] = n;
    own = before = qceil(n, G);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(ALL, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) s_base[warp] = before;
    before -= own;
  }
  __syncthreads();
  if (threadIdx.x < POP_QMOE_MAX_EXPERTS) {
    const int x = threadIdx.x;
    for (int w = 0; w < warp; ++w) before += s_base[w];
#pragma unroll
    for (int w = 0; w < PLAN_WARPS; ++w) s_at[w][x] += before * G;
  }
  __syncthreads();
  for (int c = p0; c < p1; c += 128) {
    if (p1 - p0 > 128) load(c, false);  // else they are still there
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + 32 * i >= p1) break;
      const unsigned same = __match_any_sync(ALL, e[i]);
      int at = 0;
      if (e[i] >= 0) at = s_at[warp][e[i]];
      __syncwarp();
      const int p = c + 32 * i + lane;
      if (p < p1) row_of[p] = e[i] < 0 ? -1 : at + __popc(same & ((1u << lane) - 1u));
      if (e[i] >= 0 && lane == __ffs(same) - 1) s_at[warp][e[i]] = at + __popc(same);
      __syncwarp();
    }
  }
}

// Four outputs per thread, up to K slots at a time so that their rows are on their way together. Bound by memory: 4096
// tokens of 4096 outputs, two slots, 29 us with 134 MB read and 34 written (5.8 TB/s).
template <int K>
__global__ void __launch_bounds__(256) k_combine(const float* __restrict__ o, const int* __restrict__ row_of,
                                                 const float* __restrict__ weights, int k, int D,
                                                 void* __restrict__ y, long long ldy, int out_f32) {
  const size_t t = blockIdx.x;
  const int d = 4 * (blockIdx.y * 256 + threadIdx.x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < k; j0 += K) {
    int r[K];
    float w[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      r[j] = j0 + j < k ? __ldcg(row_of + t * k + j0 + j) : -1;
      w[j] = r[j] >= 0 ? weights[t * k + j0 + j] : 0.f;
    }
    if (j0 == 0) {
      pdl_wait();  // the experts' outputs (the places were there before they began)
      pdl_trigger();
      if (d >= D) return;
    }
    float4 v[K];
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (r[j] >= 0) v[j] = __ldcg(reinterpret_cast<const float4*>(o + static_cast<size_t>(r[j]) * D + d));
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (r[j] < 0) continue;
      acc.x = fmaf(w[j], v[j].x, acc.x);
      acc.y = fmaf(w[j], v[j].y, acc.y);
      acc.z = fmaf(w[j], v[j].z, acc.z);
      acc.w = fmaf(w[j], v[j].w, acc.w);
    }
  }
  if (out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(y) + t * ldy + d) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + t * ldy + d) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

}  // namespace

cudaError_t launch_quantize_rows(const QRowsArgs& in, const QRowsOut& out, cudaStream_t st) {
  const int KB = qceil(in.K, QB);
  const int per = KB < 32 ? 32 / KB : 1;
  const dim3 grid(qceil(in.M, per), qceil(KB, 32));
  if (in.kind == 0) return launch_q(k_quantize_rows<0>, grid, 256, 0, st, in, out, per);
  if (in.kind == 1) return launch_q(k_quantize_rows<1>, grid, 256, 0, st, in, out, per);
  return launch_q(k_quantize_rows<2>, grid, 256, 0, st, in, out, per);
}

cudaError_t launch_pack_matrix(const void* W, const float* Ws, int N, int K, uint8_t* img, float* s, int step,
                               int part, cudaStream_t st) {
  return launch_plain(k_pack_matrix, dim3(qceil(K, QB), qceil(N, QB)), 256, st, W, Ws, N, K, img, s, step, part);
}

cudaError_t launch_plan(const int* experts, int pairs, int E, int G, int* counts, int* row_of, unsigned* err,
                        cudaStream_t st) {
  return launch_q(k_plan, dim3(1), 32 * PLAN_WARPS, 0, st, experts, pairs, E, G, counts, row_of, err);
}

cudaError_t launch_combine(const float* o, const int* row_of, const float* weights, int T, int k, int D, void* y,
                           long long ldy, int out_f32, cudaStream_t st) {
  const dim3 grid(T, qceil(D, 1024));
  if (k <= 2) return launch_q(k_combine<2>, grid, 256, 0, st, o, row_of, weights, k, D, y, ldy, out_f32);
  return launch_q(k_combine<4>, grid, 256, 0, st, o, row_of, weights, k, D, y, ldy, out_f32);
}

}  // namespace pop
