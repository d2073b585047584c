// Device helpers of the 8-bit operators: e4m3 rounding, bulk copies, the e4m3 tensor-core product.
#pragma once
#include <cuda_fp8.h>

#include "pop_device.cuh"
#include "pop_qinternal.h"

namespace pop {

// ------------------------------------------------------------------ e4m3
// How the values of a block with largest magnitude a become (448 * x) / a, which e4m3x2 rounds: 448 = 0.875 * 512 is
// e4m3's largest value, and the power of two of it changes no rounding (include/pop_quant.h has 0.875, whose
// product does not overflow; here a block with a > 2^100 is scaled by 2^-64 first, which is as good). The quotient
// is q0 = t * (1 / a) corrected once by its exact remainder (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990): a quotient that is an fp32 number, as every tie between two e4m3
// values is, comes out exactly.
struct BlockRatio {
  float k, a, y;
  __device__ __forceinline__ explicit BlockRatio(float amax, float top = 448.f) {
    const bool big = amax > 0x1p100f;
    k = big ? top * 0x1p-64f : top;
    a = big ? amax * 0x1p-64f : amax;
    y = __frcp_rn(a);
  }
  // of two values at a time
  __device__ __forceinline__ float2 operator()(float x0, float x1) const {
    float2 q;
    asm("{\n\t.reg .b64 x, k, a, y, t, q, r;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 k, {%4, %4};\n\tmov.b64 a, {%5, %5};\n\tmov.b64 y, {%6, %6};\n\t"
        "mul.rn.f32x2 t, x, k;\n\tmul.rn.f32x2 q, t, y;\n\tfma.rn.f32x2 r, q, a, t;\n\tfma.rn.f32x2 q, r, y, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=f"(q.x), "=f"(q.y)
        : "f"(x0), "f"(x1), "f"(k), "f"(-a), "f"(y));
    return q;
  }
};

__device__ __forceinline__ uint32_t e4m3x2(float2 v) { return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3); }

__device__ __forceinline__ uint4 e4m3x16(const float* v, const BlockRatio& ratio) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x2(ratio(v[4 * i], v[4 * i + 1])) | (e4m3x2(ratio(v[4 * i + 2], v[4 * i + 3])) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The bits of |x| are ordered as the numbers are, with NaN above infinity: a block with a NaN gets a
// NaN for its largest value.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t AMAX_MIN_BITS = 0x1f800000u;  // 2^-64

// max(m, |a|, |b|), NaN if any is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// a / 448, rounded once: the product with 1 / 448 corrected by its exact remainder, as above.
__device__ __forceinline__ float block_scale(float a) {
  constexpr float y = 1.f / 448.f;
  const float q = a * y;
  return a == INFINITY ? a : fmaf(fmaf(-q, 448.f, a), y, q);
}

// SiLU(g) u. __expf and __fdividef are off by a few units of 2^-23, far less than the e4m3 rounding of
// the result; the full-precision forms take about three times the instructions.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

// sigma(g). __expf and __fdividef are off by a few units of 2^-23; what comes of them is rounded to bf16 or int8.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// ------------------------------------------------------------------ 8-bit integers
// Eight 8-bit integers as fp16, exactly: 1024 + (128 + q) has 128 + q in its low bits.
__device__ __forceinline__ uint4 half8(uint32_t lo, uint32_t hi) {
  const auto two = [](uint32_t w, uint32_t sel) {
    uint32_t h = __byte_perm(w, 0x64646464u, sel);
    asm("sub.f16x2 %0, %0, %1;" : "+r"(h) : "r"(0x64806480u));  // 1152
    return h;
  };
  lo ^= 0x80808080u;
  hi ^= 0x80808080u;
  return make_uint4(two(lo, 0x4140), two(lo, 0x4342), two(hi, 0x4140), two(hi, 0x4342));
}

// The nearest integer to each of two quotients, as the low byte of a float's bits: 1.5 * 2^23 + q.
__device__ __forceinline__ uint2 nearest(float2 v) {
  uint64_t b;
  uint2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(v.x), "f"(v.y));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(b) : "l"(0x4b4000004b400000ull));
  asm("mov.b64 {%0, %1}, %2;" : "=r"(r.x), "=r"(r.y) : "l"(b));
  return r;
}

// ... as fp16.
__device__ __forceinline__ uint32_t half2_of(uint2 bits) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(__uint_as_float(bits.y) - 0x1.8p23f), "f"(__uint_as_float(bits.x) - 0x1.8p23f));
  return h;
}
__device__ __forceinline__ uint32_t half2_nearest(float2 v) { return half2_of(nearest(v)); }

// ------------------------------------------------------------------ launches
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class K, class... Args>
cudaError_t launch_q(K kernel, dim3 grid, int block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ copies and products
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Instruction descriptor, kind::f8f6f4 with e4m3 A and B (format 0), both K-major, and fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// A k-block (128 bytes of k) is four products of 32. a_lo and b_lo: the low words of the operands' descriptors
// (address >> 4 | leading offset), which alone change from block to block. The descriptors are put together
// here from 32-bit words: as 64-bit sums in a thread's own registers they took about 70 cycles a product to
// issue, as much as the product takes.
constexpr uint32_t DESC_LO = 1u << 16;                                 // leading byte offset 16 (not used by the swizzle)
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | DESC_LO; }
__device__ __forceinline__ void umma_block(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo + 2 * k), "r"(b_lo + 2 * k), "r"(idesc), "r"(DESC_HI), "r"(k > 0 ? 1u : 0u)
        : "memory");
}

// Waits until the phase with the given parity has completed; false after the limit, or once another role of the
// CTA has given up. These kernels wait several times per k-block: the timer is first read after a number of tries.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, QWait limit, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & limit.more) == 0u) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0)
        t0 = now;
      else if (now - t0 > limit.ns)
        return false;
    }
  }
}

// One lane of the warp (the same one every time). Code that only this lane runs inside a loop of the whole warp
// keeps its operands in uniform registers, which the tensor-core instructions need them in.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ------------------------------------------------------------------ pairs of CTAs (clusters of two)
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a barrier at the same place in the first CTA of the cluster.
__device__ __forceinline__ uint32_t first_cta(uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}
// Arrives there. Of this thread's operations it orders what the barrier's own kind orders: a copy that a
// barrier of this CTA has reported, and tensor-memory loads that tcgen05.wait::ld and a fence have ended. A
// release at cluster scope would also wait for every load still on its way.
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
// The address of the same place in a CTA of the cluster; and 16 bytes from there.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t cta) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(cta));
  return a;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_result, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_result)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// The same on both CTAs' tensor cores: A's rows and B's rows lie half in each, at the same addresses.
__device__ __forceinline__ void umma_block_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo + 2 * k), "r"(b_lo + 2 * k), "r"(idesc), "r"(DESC_HI), "r"(k > 0 ? 1u : 0u)
        : "memory");
}
// Arrives on `bar` in both CTAs once all products issued so far by this thread have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

// Waits for this thread's tensor-memory loads; r names what they fill, so that nothing reads it before.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// Barrier 1 of the block's N epilogue threads: whether `bad` holds in any of them, the same for all.
template <int N>
__device__ __forceinline__ bool epi_any(bool bad) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, r;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred r, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, r;\n\t}"
      : "=r"(any)
      : "r"(bad ? 1u : 0u), "n"(N)
      : "memory");
  return any != 0;
}

// Two fp32 fused multiply-adds: a += d * f.
__device__ __forceinline__ void fma2(float2& a, float dx, float dy, float f) {
  uint64_t v, w, s;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(dx), "f"(dy));
  asm("mov.b64 %0, {%1, %1};" : "=l"(w) : "f"(f));
  asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "f"(a.x), "f"(a.y));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(v), "l"(w));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(s));
}

// ... with a factor for each, of float bits: a += d * f; and such factors, s times (x, y).
__device__ __forceinline__ void fma2(float2& a, uint32_t dx, uint32_t dy, uint64_t f) {
  uint64_t v, s;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(dx), "r"(dy));
  asm("mov.b64 %0, {%1, %2};" : "=l"(s) : "f"(a.x), "f"(a.y));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(s) : "l"(v), "l"(f));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(s));
}
__device__ __forceinline__ uint64_t mul2(float s, float x, float y) {
  uint64_t v, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(w) : "f"(s));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
  return v;
}

// 32 bytes, aligned to 32, in one store.
__device__ __forceinline__ void st_sector(void* p, uint4 lo, uint4 hi) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w),
               "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

// ------------------------------------------------------------------ groups
// The groups of a product, in shared memory.
struct Groups {
  int tile0[POP_QMOE_MAX_EXPERTS + 1];  // first tile of each
  int count[POP_QMOE_MAX_EXPERTS];      // rows
  int run0[POP_QMOE_MAX_EXPERTS];       // first run of G rows

  // Group e has ceil(count[e] / rows) * per tiles. Returns their number; all threads of the block call it. The rows of
  // each group are given (counts), or counted here from the experts of all pairs. With BATCH four of them are on their way
  // at a time, and zero() has gone before, with a barrier of the block between the two (333 tokens through 6 of 64
  // experts: 97 us without, 96 with it). The wide product's registers do not hold that (43.2 -> 45 us, by spills).
  __device__ __forceinline__ void zero(const QGemmArgs& a) {
    if (a.experts)
      for (int e = threadIdx.x; e < a.E; e += blockDim.x) count[e] = 0;
  }
  template <bool BATCH>
  __device__ __forceinline__ int fill(const QGemmArgs& a, int rows, int per) {
    if (a.experts && BATCH) {
      for (int p0 = threadIdx.x; p0 < a.M; p0 += 4 * blockDim.x) {
        int es[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = p0 + i * static_cast<int>(blockDim.x);
          es[i] = p < a.M ? __ldg(a.experts + p) : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (static_cast<unsigned>(es[i]) < static_cast<unsigned>(a.E)) atomicAdd(&count[es[i]], 1);
      }
      __syncthreads();
    } else if (a.experts) {
      for (int e = threadIdx.x; e < a.E; e += blockDim.x) count[e] = 0;
      __syncthreads();
      for (int p = threadIdx.x; p < a.M; p += blockDim.x) {
        const int e = __ldg(a.experts + p);
        if (static_cast<unsigned>(e) < static_cast<unsigned>(a.E)) atomicAdd(&count[e], 1);
      }
      __syncthreads();
    }
    if (!a.counts && !a.experts) {
      if (threadIdx.x == 0) {
        tile0[0] = 0;
        tile0[1] = qceil(a.M, rows) * per;
        count[0] = a.M;
        run0[0] = 0;
      }
    } else if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int tiles = 0, runs = 0;
      for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        const int c = e >= a.E ? 0 : a.experts ? count[e] : __ldcg(a.counts + e);
        const int own_t = qceil(c, rows) * per, own_r = qceil(c, a.G);
        int t = own_t, r = own_r;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, t, o), v = __shfl_up_sync(0xffffffffu, r, o);
          if (lane >= o) t += u, r += v;
        }
        if (e < a.E) {
          tile0[e] = tiles + t - own_t;
          count[e] = c;
          run0[e] = runs + r - own_r;
        }
        tiles += __shfl_sync(0xffffffffu, t, 31);
        runs += __shfl_sync(0xffffffffu, r, 31);
      }
      if (lane == 0) tile0[a.E] = tiles;
    }
    __syncthreads();
    return tile0[a.E];
  }

  // The group of a tile: the last e with tile0[e] <= t (the ones without tiles come before it).
  __device__ __forceinline__ int of(int E, int t) const {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile0[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
};

// Limit of the waits in which a CTA that gives up lets its own copies and products finish (the others' is the
// handle's, QGemmArgs::wait).
constexpr QWait Q_DRAIN(1000000000ull);

}  // namespace pop
