// Rows and matrices in e4m3 with a scale per block of 128: quantising, operand images, the grouping of
// tokens by expert and the weighted sum of the experts' outputs (include/pop_quant.h, pop_qinternal.h).
#include "pop_qdevice.cuh"

namespace pop {
namespace {

__device__ __forceinline__ void unpack8(const void* p, int kind, float* v) {
  if (kind == 0) {
    const uint4 w = ldg_stream(p);
    v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
  } else {
    const uint4 a = ldg_stream(p), b = ldg_stream(static_cast<const uint8_t*>(p) + 16);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  }
}

// Eight lanes per block of 128, 16 values each.
__global__ void __launch_bounds__(256) k_quantize_rows(QRowsArgs in, QRowsOut out) {
  const int KB = qceil(in.K, QB);
  const long long units = static_cast<long long>(in.M) * KB;
  const int lane8 = threadIdx.x & 7;
  for (long long u = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
       u - ((threadIdx.x & 31) >> 3) < units; u += (static_cast<long long>(gridDim.x) * blockDim.x) >> 3) {
    const bool on = u < units;
    const int row = on ? static_cast<int>(u / KB) : 0;
    const int kb = on ? static_cast<int>(u - static_cast<long long>(row) * KB) : 0;
    const int k0 = kb * QB + lane8 * 16;
    const int n8 = on ? min(max((in.K - k0) >> 3, 0), 2) : 0;  // runs of 8 values this lane has
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    float s = 0.f;
    if (in.kind == 2) {
      const uint8_t* p = static_cast<const uint8_t*>(in.x) + static_cast<size_t>(row) * in.ldx + k0;
      if (n8 > 0) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        q.x = a.x, q.y = a.y;
      }
      if (n8 > 1) {
        const uint2 b = *reinterpret_cast<const uint2*>(p + 8);
        q.z = b.x, q.w = b.y;
      }
      if (on) s = in.xs[static_cast<size_t>(row) * in.lds + kb];
    } else {
      const int size = in.kind == 0 ? 2 : 4;
      const uint8_t* p = static_cast<const uint8_t*>(in.x) + (static_cast<size_t>(row) * in.ldx + k0) * size;
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
      if (n8 > 0) unpack8(p, in.kind, v);
      if (n8 > 1) unpack8(p + 8 * size, in.kind, v + 8);
      uint32_t m = AMAX_MIN_BITS;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, abs_bits(v[i]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float a = __uint_as_float(m);
      q = e4m3x16(v, a);
      s = __fdiv_rn(a, 448.f);
    }
    if (!on) continue;
    if (out.G == 0) {
      uint8_t* p = out.q + static_cast<size_t>(row) * out.ldq + k0;
      if (n8 > 0) *reinterpret_cast<uint2*>(p) = make_uint2(q.x, q.y);
      if (n8 > 1) *reinterpret_cast<uint2*>(p + 8) = make_uint2(q.z, q.w);
      if (lane8 == 0) out.s[static_cast<size_t>(row) * KB + kb] = s;
      continue;
    }
    for (int j = 0; j < out.k; ++j) {
      const int r = out.row_of ? out.row_of[static_cast<size_t>(row) * out.k + j] : row;
      if (r < 0) continue;
      const size_t image = (static_cast<size_t>(r / out.G) * KB + kb) * out.G * QB;
      *reinterpret_cast<uint4*>(out.q + image + image_at(r % out.G, lane8 * 16)) = q;
      if (lane8 == 0) out.s[static_cast<size_t>(kb) * out.rows + r] = s;
    }
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
      if (n8 > 0) unpack8(p, 0, v[i]);
      if (n8 > 1) unpack8(p + 16, 0, v[i] + 8);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[i][j]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_max, m);
  __syncthreads();
  const float a = __uint_as_float(s_max);
#pragma unroll
  for (int i = 0; i < 4; ++i) dst[image_at(r0 + 32 * i, c * 16) >> 4] = e4m3x16(v[i], a);
  if (threadIdx.x == 0) *scale = __fdiv_rn(a, 448.f);
}

// One CTA. Warp w numbers the pairs of experts w, w + 32, ... in ascending order, a ballot per 32 pairs;
// then the runs' prefix sums; then every pair's row.
__global__ void __launch_bounds__(1024) k_plan(const int* __restrict__ experts, int pairs, int E, int G,
                                               int* __restrict__ counts, int* __restrict__ run0,
                                               int* __restrict__ row_of, unsigned* __restrict__ err) {
  __shared__ int s_run0[POP_QMOE_MAX_EXPERTS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned lt = (1u << lane) - 1u;
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    const int e = experts[p];
    if (e < 0 || e >= E) {
      row_of[p] = -1;
      if (e != -1) atomicOr(err, QERR_EXPERT);
    }
  }
  for (int e = warp; e < E; e += blockDim.x >> 5) {
    int base = 0;
    for (int c = 0; c < pairs; c += 32) {
      const bool hit = c + lane < pairs && experts[c + lane] == e;
      const unsigned m = __ballot_sync(0xffffffffu, hit);
      if (hit) row_of[c + lane] = base + __popc(m & lt);
      base += __popc(m);
    }
    if (lane == 0) counts[e] = base;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int s = 0;
    for (int e = 0; e < E; ++e) {
      s_run0[e] = s;
      run0[e] = s;
      s += qceil(counts[e], G);
    }
    run0[E] = s;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    const int e = experts[p];
    if (e >= 0 && e < E) row_of[p] += s_run0[e] * G;
  }
}

// Four outputs per thread.
__global__ void __launch_bounds__(256) k_combine(const float* __restrict__ o, const int* __restrict__ row_of,
                                                 const float* __restrict__ weights, int k, int D,
                                                 void* __restrict__ y, long long ldy, int out_f32) {
  const size_t t = blockIdx.x;
  const int d = 4 * (blockIdx.y * 256 + threadIdx.x);
  if (d >= D) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < k; ++j) {
    const int r = row_of[t * k + j];
    if (r < 0) continue;
    const float w = weights[t * k + j];
    const float4 v = *reinterpret_cast<const float4*>(o + static_cast<size_t>(r) * D + d);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  if (out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(y) + t * ldy + d) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + t * ldy + d) =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

}  // namespace

cudaError_t launch_quantize_rows(const QRowsArgs& in, const QRowsOut& out, cudaStream_t st) {
  const long long threads = static_cast<long long>(in.M) * qceil(in.K, QB) * 8;
  const long long grid = (threads + 255) / 256;
  k_quantize_rows<<<static_cast<unsigned>(grid < (1ll << 30) ? grid : (1ll << 30)), 256, 0, st>>>(in, out);
  return cudaGetLastError();
}

cudaError_t launch_pack_matrix(const void* W, const float* Ws, int N, int K, uint8_t* img, float* s, int step,
                               int part, cudaStream_t st) {
  k_pack_matrix<<<dim3(qceil(K, QB), qceil(N, QB)), 256, 0, st>>>(W, Ws, N, K, img, s, step, part);
  return cudaGetLastError();
}

cudaError_t launch_plan(const int* experts, int pairs, int E, int G, int* counts, int* run0, int* row_of,
                        unsigned* err, cudaStream_t st) {
  k_plan<<<1, 1024, 0, st>>>(experts, pairs, E, G, counts, run0, row_of, err);
  return cudaGetLastError();
}

cudaError_t launch_combine(const float* o, const int* row_of, const float* weights, int T, int k, int D, void* y,
                           long long ldy, int out_f32, cudaStream_t st) {
  k_combine<<<dim3(T, qceil(D, 1024)), 256, 0, st>>>(o, row_of, weights, k, D, y, ldy, out_f32);
  return cudaGetLastError();
}

}  // namespace pop
