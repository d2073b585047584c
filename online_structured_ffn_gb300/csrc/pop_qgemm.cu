// Products of rows and matrices in e4m3 with block scales (pop_qinternal.h): a tile of 16 rows by 128
// outputs per CTA on the CUDA cores.
#include <cuda_fp8.h>

#include "pop_device.cuh"
#include "pop_qinternal.h"

namespace pop {
namespace {

constexpr int RT = 16;

__device__ __forceinline__ float e4m3_f(uint8_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(b, __NV_E4M3);
  return __half2float(__half(h));
}

template <bool GATED>
__global__ void __launch_bounds__(256) k_qgemm(QGemmArgs a) {
  constexpr int P = GATED ? 2 : 1;
  __shared__ float s_x[RT][QB];
  __shared__ float s_s[RT];
  __shared__ uint32_t s_max[RT];
  const int KB = qceil(a.K, QB), NT = qceil(a.N, QB);
  const int n = threadIdx.x & 127, half = threadIdx.x >> 7;  // output n of the tile, rows 8 half .. + 8
  const int t = blockIdx.x;
  int e = 0, tile = blockIdx.y, cnt = a.counts ? a.counts[0] : a.M;
  while (tile >= qceil(cnt, RT)) {
    tile -= qceil(cnt, RT);
    if (++e >= a.E) return;
    cnt = a.counts[e];
  }
  const int row0 = (a.run0 ? a.run0[e] : 0) * a.G + tile * RT;
  const int rows = min(RT, cnt - tile * RT);
  const uint8_t* w = a.w + e * a.w_stride;
  const float* ws = a.ws + e * a.ws_stride;
  float acc[P][8];
  for (int p = 0; p < P; ++p)
    for (int i = 0; i < 8; ++i) acc[p][i] = 0.f;
  for (int kb = 0; kb < KB; ++kb) {
    __syncthreads();
    for (int i = threadIdx.x; i < RT * QB; i += 256) {
      const int r = i >> 7, k = i & 127, g = row0 + r;
      s_x[r][k] = e4m3_f(a.act[(static_cast<size_t>(g / a.G) * KB + kb) * a.G * QB + image_at(g % a.G, k)]);
    }
    if (threadIdx.x < RT) s_s[threadIdx.x] = a.act_s[static_cast<size_t>(kb) * a.rows + row0 + threadIdx.x];
    __syncthreads();
    for (int p = 0; p < P; ++p) {
      const size_t slot = (static_cast<size_t>(t) * KB + kb) * P + p;
      float part[8];
      for (int i = 0; i < 8; ++i) part[i] = 0.f;
      for (int k = 0; k < QB; ++k) {
        const float v = e4m3_f(w[slot * QTILE + image_at(n, k)]);
        for (int i = 0; i < 8; ++i) part[i] = fmaf(v, s_x[8 * half + i][k], part[i]);
      }
      const float sw = ws[slot];
      for (int i = 0; i < 8; ++i) acc[p][i] = fmaf(sw * s_s[8 * half + i], part[i], acc[p][i]);
    }
  }
  const int col = t * QB + n;
  if (!GATED) {
    for (int i = 0; i < 8; ++i) {
      if (8 * half + i >= rows || col >= a.N) continue;
      const size_t o = static_cast<size_t>(row0 + 8 * half + i) * a.ldy + col;
      if (a.out_f32)
        static_cast<float*>(a.y)[o] = acc[0][i];
      else
        static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(acc[0][i]);
    }
    return;
  }
  if (threadIdx.x < RT) s_max[threadIdx.x] = 0x1f800000u;
  __syncthreads();
  for (int i = 0; i < 8; ++i) {
    const float g = acc[0][i];
    acc[0][i] = g / (1.f + expf(-g)) * acc[P - 1][i];
    atomicMax(&s_max[8 * half + i], __float_as_uint(acc[0][i]) & 0x7fffffffu);
  }
  __syncthreads();
  for (int i = 0; i < 8; ++i) {
    const int g = row0 + 8 * half + i;
    if (8 * half + i >= rows) continue;
    const float m = __uint_as_float(s_max[8 * half + i]);
    const float q = 512.f * __fdiv_rn(0.875f * acc[0][i], m);
    a.h[(static_cast<size_t>(g / a.G) * NT + t) * a.G * QB + image_at(g % a.G, n)] =
        __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    if (n == 0) a.h_s[static_cast<size_t>(t) * a.rows + g] = __fdiv_rn(m, 448.f);
  }
}

}  // namespace

cudaError_t launch_qgemm(const QGemmArgs& a, bool gated, cudaStream_t st) {
  const int tiles = qceil(a.M, RT) + (a.counts ? (a.E < a.M ? a.E : a.M) : 0);
  const dim3 grid(qceil(a.N, QB), tiles);
  if (gated)
    k_qgemm<true><<<grid, 256, 0, st>>>(a);
  else
    k_qgemm<false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pop
