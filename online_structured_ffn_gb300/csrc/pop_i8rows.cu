// Rows and matrices in 8-bit integers: quantising with a scale per row, the fp16 rows that the products take, the matrix
// images (include/pop_int8.h, pop_i8.h).
#include "pop_i8.h"
#include "pop_qdevice.cuh"

namespace pop {
namespace {

// 16 bytes that are read once. Not through the read-only path: this kernel starts before the one in front has ended, which may
// be writing them.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

template <bool F32>
struct Piece {
  static constexpr int V = F32 ? 4 : 8;  // values
  float v[V];
  __device__ __forceinline__ explicit Piece(const uint4& w) {
    if constexpr (F32) {
      v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
    } else {
      v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
      v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
    }
  }
  __device__ __forceinline__ float most(float m) const {
#pragma unroll
    for (int j = 0; j < V; j += 2) m = max_abs(m, v[j], v[j + 1]);
    return m;
  }
};

// T threads to a row, which hold HELD pieces of 16 bytes each between the two passes over it, a CTA of 256 (or T, if that is
// more) threads. A row's values stay in registers, as they stand in memory, between the pass for the largest and the one that
// rounds; of rows longer than HELD pieces a thread the rest is read again.
// Bound by memory, with the row's largest in the way: 4096 x 4096 of bf16 9.8 us (5.1 TB/s read and written), 1001 x 11008 of
// float32 11.3 (4.9), 16,384 x 1024 of bf16 9.3 (5.4).
template <int T, int HELD, bool F32>
__global__ void __launch_bounds__(T > 256 ? T : 256, (HELD > 4 ? 1024 : 1536) / (T > 256 ? T : 256)) k_i8_rows(const __grid_constant__ I8RowsArgs a) {
  constexpr int ROWS = T > 256 ? 1 : 256 / T, WARPS = T / 32, V = Piece<F32>::V;
  __shared__ float s_most[ROWS][WARPS];
  const int t = threadIdx.x % T, in = threadIdx.x / T;
  const long long row = static_cast<long long>(blockIdx.x) * ROWS + in;
  pdl_wait();
  pdl_trigger();
  const bool on = row < a.M;
  const int n = on ? a.K / V : 0;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + (on ? row : 0) * a.ldx * (F32 ? 4 : 2));
  uint4 held[HELD];
#pragma unroll
  for (int h = 0; h < HELD; ++h) held[h] = t + h * T < n ? ld_stream(x + t + h * T) : make_uint4(0u, 0u, 0u, 0u);
  float most = __uint_as_float(AMAX_MIN_BITS);
  if (a.amax) {
    for (int i = a.parts > 1 ? t : 0; on && i < a.parts; i += a.parts > 1 ? T : 1)
      most = max_abs(most, __uint_as_float(__ldcg(a.amax + static_cast<size_t>(i) * THIN16_MOST + row)), 0.f);
  } else {
#pragma unroll
    for (int h = 0; h < HELD; ++h) most = Piece<F32>(held[h]).most(most);
    for (int i = t + HELD * T; i < n; i += T) most = Piece<F32>(ld_stream(x + i)).most(most);
  }
  if (!a.amax || a.parts > 1) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) most = max_abs(most, __shfl_xor_sync(0xffffffffu, most, o), 0.f);
    if (WARPS > 1) {
      if ((t & 31) == 0) s_most[in][t >> 5] = most;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WARPS; ++w) most = max_abs(most, s_most[in][w], 0.f);
    }
  }
  if (!on) return;
  const bool finite = most < INFINITY;
  const BlockRatio ratio(finite ? most : 1.f, 127.f);
  const auto put = [&](int i, const uint4& w) {
    const Piece<F32> e(w);
    uint2 r[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) r[j] = finite ? nearest(ratio(e.v[2 * j], e.v[2 * j + 1])) : make_uint2(0x4b400000u, 0x4b400000u);
    uint32_t o[V / 2];
    if (a.q) {
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        o[j] = __byte_perm(__byte_perm(r[2 * j].x, r[2 * j].y, 0x0040), __byte_perm(r[2 * j + 1].x, r[2 * j + 1].y, 0x0040), 0x5410);
      uint32_t* q = reinterpret_cast<uint32_t*>(a.q + row * a.ldq + V * i);
      if constexpr (F32)
        *q = o[0];
      else
        *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) o[j] = half2_of(r[j]);
      uint32_t* q = reinterpret_cast<uint32_t*>(a.half + row * a.K + V * i);
      if constexpr (F32)
        *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
      else
        *reinterpret_cast<uint4*>(q) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  };
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if (t + h * T < n) put(t + h * T, held[h]);
  for (int i = t + HELD * T; i < n; i += T) put(i, ld_stream(x + i));
  if (t == 0) {
    a.s[row] = finite ? __fdiv_rn(most, 127.f) : __uint_as_float(0x7fffffffu);
    if (a.clear) a.clear[row] = 0u;
  }
}

__global__ void __launch_bounds__(256) k_i8_half(const int8_t* q, long long ldq, const float* s, int K, uint16_t* half, float* sx) {
  pdl_wait();
  pdl_trigger();
  const size_t row = blockIdx.x;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < K >> 3; i += 256 * gridDim.y) {
    const uint2 w = __ldcg(reinterpret_cast<const uint2*>(q + row * ldq + 8 * i));
    *reinterpret_cast<uint4*>(half + row * K + 8 * i) = half8(w.x, w.y);
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) sx[row] = __ldcg(s + row);
}

// A CTA per block: two pieces of 16 bytes a thread.
__global__ void __launch_bounds__(256) k_i8_pack(const int8_t* __restrict__ W, int N, int K, uint8_t* __restrict__ image) {
  const size_t block = static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  const int r = threadIdx.x & 127, row = blockIdx.y * 128 + r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = (threadIdx.x >> 7) + 2 * i, k = blockIdx.x * 64 + 16 * j;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const int8_t* p = W + static_cast<size_t>(row) * K + k;
    if (row < N && k < K) {
      const uint2 lo = *reinterpret_cast<const uint2*>(p);
      v.x = lo.x, v.y = lo.y;
    }
    if (row < N && k + 8 < K) {
      const uint2 hi = *reinterpret_cast<const uint2*>(p + 8);
      v.z = hi.x, v.w = hi.y;
    }
    reinterpret_cast<uint4*>(image + block * W8_BLOCK)[j * 128 + r] = v;
  }
}

template <int T, int HELD>
cudaError_t rows(const I8RowsArgs& a, cudaStream_t st) {
  constexpr int ROWS = T > 256 ? 1 : 256 / T, BLOCK = T > 256 ? T : 256;
  const dim3 grid(static_cast<unsigned>(qceil(a.M, ROWS)));
  return a.f32 ? launch_q(k_i8_rows<T, HELD, true>, grid, BLOCK, 0, st, a) : launch_q(k_i8_rows<T, HELD, false>, grid, BLOCK, 0, st, a);
}

}  // namespace

cudaError_t launch_i8_rows(const I8RowsArgs& a, cudaStream_t st) {
  const int pieces = a.K / (a.f32 ? 4 : 8);
  // As few threads as hold the row in eight pieces each: the sum over a CTA's warps costs more than the longer threads. (us with 64
  // threads and eight, 128 and four, 128 and eight: 4096 rows of 512 pieces 9.8, 10.0, 11.6; 1000 of them 3.9, 4.7, 3.8; 2048 of
  // 2048, with 256 and eight, 512 and four, 512 and eight: 12.4, 14.2, 17.4.)
  if (pieces <= 32 * 4) return rows<32, 4>(a, st);
  if (pieces <= 32 * 8) return rows<32, 8>(a, st);
  if (pieces <= 64 * 8) return rows<64, 8>(a, st);
  if (pieces <= 128 * 8) return rows<128, 8>(a, st);
  return pieces <= 256 * 8 ? rows<256, 8>(a, st) : rows<512, 8>(a, st);
}

cudaError_t launch_i8_half(const int8_t* q, long long ldq, const float* s, int M, int K, uint16_t* half, float* sx, cudaStream_t st) {
  return launch_q(k_i8_half, dim3(M, qceil(K, 4096)), 256, 0, st, q, ldq, s, K, half, sx);
}

cudaError_t launch_i8_pack(const int8_t* W, int N, int K, uint8_t* image, cudaStream_t st) {
  return launch_plain(k_i8_pack, dim3(qceil(K, 64), qceil(N, 128)), 256, st, W, N, K, image);
}

}  // namespace pop
