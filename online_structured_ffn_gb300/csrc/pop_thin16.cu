// Products of few rows (tokens) and a matrix of bf16 or of 8-bit integers (pop_wide16.h): the matrix streams once.
//
// The matrix is the M operand, 128 of its rows a tile (gated: of gate and of up), the tokens the N operand, NT = 16, 32, 64
// or 128 of them. A tile is given to a cluster of S CTAs, which take a run of the k-blocks each, as many as let all SMs
// stream at once; then each has 1 / S of the tokens: it reads the others' parts of them from their shared memory, adds
// them in the order of k and has their epilogue.
//
// Backward the matrix is multiplied by its other side: its blocks come as two boxes of 64 values by 64 k and the tensor cores
// read them mn-major. The gradient of the rows is the sum of two such products, one after the other in k; that of the hidden
// values goes on to the gate's and the up's in the epilogue.
//
// 8-bit integers: a block of 128 rows by 64 k comes as it is; 128 threads read a row each, turn it into fp16 and put it into
// tensor memory, from where the product takes it. (In shared memory the fp16 block would be written and read once more.)
//
// Up to 16 rows, where a CTA's k-blocks of them fit beside the ring, need no kernel before this one that quantises (or widens)
// them: every CTA brings its own from bf16, float32 or integers into their fp16 operands while the matrix's first blocks are on
// their way. The rows' largest magnitudes, which bf16 rows need first, it finds for itself; a gated MLP's hidden rows come
// with those of each tile of channels. (Two warps that converted each stage's rows as they came took 0.4 us a k-block,
// longer than its matrix takes.)
//
// Bound by the matrix's bytes, and with short ones by what comes before and after them (some 5 us: first bytes 1.2, the
// cluster's meeting 1.2, the others' parts 0.7, its end 1). Back to back: gate and up and down of one token, bf16 46 us for 270
// MB (5.9 TB/s); 8-bit: 16 rows by 8192 x 28672 with their quantising 44 us (5.4), one row by 11008 x 4096 11.4 (4.0).
//
// Warp 0: copies; the matrix's first stages go out before the kernel before this one has ended, where that does not write them.
// Warp 1: products. Warps 4..11: conversion, then the epilogue. Every wait has a limit; a CTA that gives up records
// WERR_TIMEOUT, lets its copies and products finish, frees TMEM and returns.
#include <algorithm>
#include <atomic>

#include "pop_qdevice.cuh"
#include "pop_wide16.h"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int THREADS = 384;
constexpr int BM = 128, BK = 64;
constexpr int MAX_STAGES = 8;
constexpr uint32_t BOX_MN = 64 * 64 * 2;  // one of the two boxes of a matrix that has its outputs' side contiguous
constexpr int NA = 4;  // blocks in tensor memory, of 32 columns

enum Back { FORWARD, DHIDDEN, DROWS };  // not a gradient; of the hidden values (W_DGATED), of the rows (W_DX)

template <bool I8_, bool GATED_, int NT_, bool CONV_ = false, Back BACK_ = FORWARD>
struct Thin {
  static constexpr bool I8 = I8_, GATED = GATED_;
  static constexpr Back BACK = BACK_;
  static constexpr bool MN = BACK != FORWARD;               // the matrix has its outputs' side contiguous
  static constexpr int SEGMENTS = BACK == DROWS ? 2 : 1;  // products that are added
  static constexpr bool CONV = CONV_;  // the rows are converted on the way
  static constexpr int NT = NT_, P = GATED ? 2 : 1;
  static constexpr int PER_SM = NT <= 64 ? 2 : 1;
  static constexpr uint32_t W_BYTES = I8 ? W8_BLOCK : BM * BK * 2, X_BYTES = NT * BK * 2;
  // converted rows lie behind the ring, all k-blocks of this CTA
  static constexpr uint32_t X_OFF = P * W_BYTES, STAGE = X_OFF + (CONV ? 0 : X_BYTES);
  static constexpr uint32_t KEPT = CONV ? THIN16_KEPT * X_BYTES : 0;
  static constexpr uint32_t BUDGET = (PER_SM == 2 ? 108 : 216) * 1024 - KEPT;
  static constexpr int FIT = BUDGET / STAGE;
  // A stage's block is converted by the same four warps every time (two sets of them take turns, plain: block by block), as one
  // that looks at a stage for the first time cannot tell a block that has not landed from the one before it; copies may land
  // out of order.
  static constexpr int STAGES = (FIT < MAX_STAGES ? FIT : MAX_STAGES) & (I8 && !GATED ? ~1 : ~0);
  static constexpr int COLS = P * NT + (I8 ? NA * 32 : 0);
  static constexpr uint32_t TMEM_COLS = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(TMEM_COLS * PER_SM <= 512, "tensor memory of an SM");
  static_assert(STAGE % 1024 == 0 && STAGES * STAGE >= P * NT * BM * 4, "a part fits into the ring");
  static constexpr uint32_t SMEM = STAGES * STAGE + KEPT + 1024;
};

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t xfull;
  uint64_t afull[NA], aempty[NA];
  uint64_t tfull;
  uint32_t tmem_base;
  int abort_flag;
  unsigned most[THIN16_MOST];   // converted rows: bits of their largest magnitude
  unsigned hmost[THIN16_MOST];  // gated: of this CTA's tokens' outputs
};

// kind::f16, A in tensor memory: a lane is a row, a column two values of k. A k-block is four products of 16.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool first) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem + 8 * k), "r"(b_lo + 2 * k), "r"(idesc), "r"(DESC_HI), "r"(k > 0 || !first ? 1u : 0u)
        : "memory");
}
// ... and both in shared memory; a matrix with its outputs' side contiguous: two boxes of 64 by 64 k, 16 rows on.
template <bool A_MN>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool first) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo + (A_MN ? 128 : 2) * k), "r"(b_lo + 2 * k), "r"(idesc), "r"(DESC_HI), "r"(k > 0 || !first ? 1u : 0u)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint4 (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w), "r"(v[2].x), "r"(v[2].y),
      "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y), "r"(v[3].z), "r"(v[3].w), "r"(v[4].x), "r"(v[4].y), "r"(v[4].z), "r"(v[4].w),
      "r"(v[5].x), "r"(v[5].y), "r"(v[5].z), "r"(v[5].w), "r"(v[6].x), "r"(v[6].y), "r"(v[6].z), "r"(v[6].w), "r"(v[7].x), "r"(v[7].y),
      "r"(v[7].z), "r"(v[7].w)
      : "memory");
}

// Eight values of a row as they stand in memory (bf16: lo alone), and quantised, as fp16.
struct Raw {
  uint4 lo, hi;
};
__device__ __forceinline__ uint4 half_of(const Raw& w, int size, bool finite, const BlockRatio& ratio) {
  float v[8];
  if (size == 2) {
    v[0] = bf16lo(w.lo.x), v[1] = bf16hi(w.lo.x), v[2] = bf16lo(w.lo.y), v[3] = bf16hi(w.lo.y);
    v[4] = bf16lo(w.lo.z), v[5] = bf16hi(w.lo.z), v[6] = bf16lo(w.lo.w), v[7] = bf16hi(w.lo.w);
  } else {
    v[0] = __uint_as_float(w.lo.x), v[1] = __uint_as_float(w.lo.y), v[2] = __uint_as_float(w.lo.z), v[3] = __uint_as_float(w.lo.w);
    v[4] = __uint_as_float(w.hi.x), v[5] = __uint_as_float(w.hi.y), v[6] = __uint_as_float(w.hi.z), v[7] = __uint_as_float(w.hi.w);
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = finite ? half2_nearest(ratio(v[2 * j], v[2 * j + 1])) : 0u;
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Barrier 2 of the eight warps.
__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 2, 256;" ::: "memory"); }

template <class T>
__global__ void __launch_bounds__(THREADS, T::PER_SM) k_thin16(const __grid_constant__ WArgs a) {
  constexpr int STAGES = T::STAGES, NT = T::NT, P = T::P;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl.abort_flag;
  const int rank = static_cast<int>(cluster_rank()), S = static_cast<int>(cluster_ctas());
  const int tile = blockIdx.x / S;
  const int KB = a.kb * T::SEGMENTS, kb0 = KB * rank / S, n = KB * (rank + 1) / S - kb0;  // this CTA's k-blocks

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1 + (T::I8 ? 4 * P : 0));
    }
    for (int i = 0; i < NA; ++i) {
      mbar_init(&ctl.afull[i], 4);
      mbar_init(&ctl.aempty[i], 1);
    }
    mbar_init(&ctl.tfull, 1);
    mbar_init(&ctl.xfull, 8);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < NT && T::I8; i += THREADS) {
    ctl.most[i] = AMAX_MIN_BITS;
    ctl.hmost[i] = 0u;
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem_base, T::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base, a_base = tmem_base + P * NT;

  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      atomicOr(a.err, WERR_TIMEOUT);
    }
  };

  // The epilogue's: a channel each lane; of the tokens, AT_ONCE at a time, either half of the warps in turn has every (2 S)-th, or
  // AT_ONCE neighbours, whose kept words are 16 bytes.
  constexpr int AT_ONCE = 4;
  const int M = a.m[0], N = a.n[0], q = warp & 3, half = (warp - 4) >> 2, r = 32 * q + lane, ch = tile * BM + r;
  constexpr bool KEEPS = T::BACK == DHIDDEN || (T::GATED && !T::I8);
  const int first = (rank + S * half) * (KEEPS ? AT_ONCE : 1), apart = KEEPS ? 1 : 2 * S;
  uint4 next[3];  // W_DGATED: kept gate and up values of two channels, of which this lane's is one
  const auto load_kept = [&](int t0) {
    if (T::BACK != DHIDDEN || t0 >= M || ch >= N) return;
    const uint32_t* k = a.saved + (static_cast<size_t>(t0 >> 5) * (N >> 1) + (ch >> 1)) * 96 + (t0 & 31);
#pragma unroll
    for (int i = 0; i < 3; ++i) next[i] = __ldcg(reinterpret_cast<const uint4*>(k) + 8 * i);
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- copies (one thread)
      const auto matrix = [&](int i, int s) {
        const int second = T::SEGMENTS == 2 && kb0 + i >= a.kb, k = (kb0 + i - (second ? a.kb : 0)) * BK;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          uint8_t* to = smem + s * T::STAGE + p * T::W_BYTES;
          if (T::I8)
            bulk_load(to, a.w8[p] + (static_cast<size_t>(tile) * a.kb + kb0 + i) * W8_BLOCK, W8_BLOCK, &ctl.full[s]);
          else if (T::MN) {
            tma_load_2d(to, &a.map[second ? 3 : 1], &ctl.full[s], tile * BM, k);
            tma_load_2d(to + BOX_MN, &a.map[second ? 3 : 1], &ctl.full[s], tile * BM + 64, k);
          } else
            tma_load_2d(to, &a.map[1 + p], &ctl.full[s], k, tile * BM);
        }
      };
      const auto rows = [&](int i, int s) {
        const int second = T::SEGMENTS == 2 && kb0 + i >= a.kb, k = (kb0 + i - (second ? a.kb : 0)) * BK;
        tma_load_2d(smem + s * T::STAGE + T::X_OFF, &a.map[second ? 2 : 0], &ctl.full[s], k, 0);
      };
      int early = T::I8 || a.b_early ? min(STAGES, n) : 0;
      for (int i = 0; i < early; ++i) {
        mbar_arrive_expect_tx(&ctl.full[i], T::STAGE);
        matrix(i, i);
      }
      if (!T::CONV) pdl_wait();
      uint32_t s = 0, phase = 1;
      int issued = 0;
      for (; issued < n; ++issued) {
        if (!mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag)) {
          fail();
          break;
        }
        if (issued >= early) {
          mbar_arrive_expect_tx(&ctl.full[s], T::STAGE);
          matrix(issued, s);
        }
        if (!T::CONV) rows(issued, s);
        if (++s == STAGES) s = 0, phase ^= 1;
      }
      // no copy of this CTA may be in flight when it exits
      for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.full[i % STAGES], (i / STAGES) & 1, Q_DRAIN, &never)) fail();
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    const bool leader = elect_one();
    constexpr uint32_t IDESC = idesc_bf16_f32(BM, NT, false, T::MN) & ~(T::I8 ? (1u << 7) | (1u << 10) : 0u);
    const uint32_t w0 = T::MN ? desc_lo(smem_u32(smem)) & 0x3fffu | (BOX_MN >> 4) << 16 : desc_lo(smem_u32(smem));
    const uint32_t x0 = desc_lo(smem_u32(smem) + (T::CONV ? STAGES * T::STAGE : T::X_OFF));
    uint32_t s = 0, phase = 0, b = 0, bphase = 0;
    bool ok = !T::CONV || mbar_wait(&ctl.xfull, 0, a.wait, abort_flag);
    for (int i = 0; i < n && ok; ++i) {
      const uint32_t x = x0 + (T::CONV ? i * T::X_BYTES : s * T::STAGE) / 16;
      ok = mbar_wait(&ctl.full[s], phase, a.wait, abort_flag);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (T::I8) ok = ok && mbar_wait(&ctl.afull[b], bphase, a.wait, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          if (T::I8) {
            umma_ts(tmem_base + p * NT, a_base + b * 32, x, IDESC, i == 0);
            umma_commit(&ctl.aempty[b]);
          } else {
            umma_ss<T::MN>(tmem_base + p * NT, w0 + (s * T::STAGE + p * T::W_BYTES >> 4), x, IDESC, i == 0);
          }
          if (p == P - 1) umma_commit(&ctl.empty[s]);
        }
        __syncwarp();
        if (T::I8 && ++b == NA) b = 0, bphase ^= 1;
      }
      if (++s == STAGES) s = 0, phase ^= 1;
    }
    if (!ok && leader) fail();
    // (also what the end of the products is waited for with, whatever has become of them)
    if (leader) umma_commit(&ctl.tfull);
    volatile int never = 0;
    if (!mbar_wait(&ctl.tfull, 0, Q_DRAIN, &never) && leader) fail();
    __syncwarp();
  } else if (warp >= 4) {
    bool ok = true;
    if constexpr (T::CONV) {
      // ---------------------------------------------------------- rows: their largest magnitudes, then their values
      pdl_wait();
      const int t = threadIdx.x - 128;
      if (a.convert == 1) {
        const int w = warp - 4, share = M >= 8 ? 1 : M >= 4 ? 2 : M >= 2 ? 4 : 8;  // warps to a row
        const int pieces = a.k >> 3, step = 32 * share;
        for (int row = w / share; row < M; row += 8 / share) {
          const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.rows) + static_cast<size_t>(row) * a.ld_rows);
          float most = 0.f;
          for (int i = (w % share) * 32 + lane; i < pieces; i += 8 * step) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = i + j * step < pieces ? __ldcg(x + i + j * step) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              most = max_abs(most, bf16lo(v[j].x), bf16hi(v[j].x));
              most = max_abs(most, bf16lo(v[j].y), bf16hi(v[j].y));
              most = max_abs(most, bf16lo(v[j].z), bf16hi(v[j].z));
              most = max_abs(most, bf16lo(v[j].w), bf16hi(v[j].w));
            }
          }
          const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));  // (NaN is above all)
          if (lane == 0) atomicMax(&ctl.most[row], bits);
        }
        rows_sync();
      } else if (a.convert == 2) {
        const int row = t & 15;
        unsigned most = 0u;
        if (row < M)
          for (int i = t >> 4; i < a.tiles_max; i += 8 * 16) {
            unsigned v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[j] = i + 16 * j < a.tiles_max ? __ldcg(a.row_max + static_cast<size_t>(i + 16 * j) * THIN16_MOST + row) : 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max(most, v[j]);
          }
        if (row < M) atomicMax(&ctl.most[row], most);
        rows_sync();
      }
      const int size = a.convert == 1 ? 2 : a.convert == 2 ? 4 : 1;
      const int row_pieces = 8 * n;  // of eight values
      uint8_t* kept = smem + STAGES * T::STAGE;
      // Four pieces a thread on their way, of whatever rows. (What the rows past the last hold goes into their own sums alone.)
      constexpr int AT_A_TIME = 4;
      for (int i0 = t; i0 < M * row_pieces; i0 += 256 * AT_A_TIME) {
        Raw v[AT_A_TIME];
        int row[AT_A_TIME], piece[AT_A_TIME];
#pragma unroll
        for (int j = 0; j < AT_A_TIME; ++j) {
          const int i = i0 + 256 * j;
          row[j] = i / row_pieces;
          piece[j] = i - row[j] * row_pieces;
          v[j].lo = v[j].hi = make_uint4(0u, 0u, 0u, 0u);
          if (row[j] >= M || kb0 * BK + 8 * piece[j] >= a.k) continue;
          const uint8_t* p = static_cast<const uint8_t*>(a.rows) + (static_cast<size_t>(row[j]) * a.ld_rows + kb0 * BK + 8 * piece[j]) * size;
          if (size == 1) {
            const uint2 w = __ldcg(reinterpret_cast<const uint2*>(p));
            v[j].lo.x = w.x, v[j].lo.y = w.y;
          } else {
            v[j].lo = __ldcg(reinterpret_cast<const uint4*>(p));
            if (size == 4) v[j].hi = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
          }
        }
#pragma unroll
        for (int j = 0; j < AT_A_TIME; ++j) {
          if (row[j] >= M) break;
          uint4 w;
          if (size == 1) {
            w = half8(v[j].lo.x, v[j].lo.y);
          } else {
            const float most = __uint_as_float(ctl.most[row[j]]);
            const bool finite = most < INFINITY;
            w = half_of(v[j], size, finite, BlockRatio(finite ? most : 1.f, 127.f));
          }
          *reinterpret_cast<uint4*>(kept + (piece[j] >> 3) * T::X_BYTES + row[j] * 128 + (((piece[j] & 7) ^ (row[j] & 7)) << 4)) = w;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.xfull);
    }
    if (T::I8) {
      // ---------------------------------------------------------- conversion: every other block, a row each thread
      uint32_t b = half, bphase = 1;
      for (int i = half; i < n * P && ok; i += 2) {
        const int stage = i / P, s = stage % STAGES;
        ok = mbar_wait(&ctl.full[s], (stage / STAGES) & 1, a.wait, abort_flag);
        const uint4* from = reinterpret_cast<const uint4*>(smem + s * T::STAGE + (i % P) * W8_BLOCK) + r;
        uint4 v[4], w[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = from[j * BM];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[2 * j] = half8(v[j].x, v[j].y);
          w[2 * j + 1] = half8(v[j].z, v[j].w);
        }
        ok = ok && mbar_wait(&ctl.aempty[b], bphase, a.wait, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) fail();
          break;
        }
        if (lane == 0) mbar_arrive(&ctl.empty[s]);
        tc_fence_after();
        tmem_st32(a_base + b * 32 + (static_cast<uint32_t>(32 * q) << 16), w);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.afull[b]);
        b ^= 2u;
        if (b < 2) bphase ^= 1;
      }
    }
    // ------------------------------------------------------------ this CTA's part: [column][row]
    pdl_wait();  // what this kernel writes may still be read by the one before
    pdl_trigger();
    load_kept(first);
    ok = ok && mbar_wait(&ctl.tfull, 0, a.wait, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) fail();
    tc_fence_after();
    float* part = reinterpret_cast<float*>(smem) + r;
    if (ok) {
#pragma unroll 1
      for (int c = 16 * half; c < P * NT; c += 32) {
        if ((c & (NT - 1)) >= a.m[0]) continue;
        uint32_t v[16];
        tmem_load(tmem_base + (static_cast<uint32_t>(32 * q) << 16) + c, v);
        tmem_wait(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * BM] = __uint_as_float(v[j]);
      }
    }
  }
  // ------------------------------------------------------------ epilogue
  const bool is = ch < N;
  float sw = 1.f, sw1 = 1.f, sx_own = 0.f;  // sx_own: of the lane-th of this warp's tokens
  if (T::I8 && warp >= 4) {
    if (is) {
      sw = __ldg(a.sw + ch);
      if (T::GATED) sw1 = __ldg(a.sw1 + ch);
    }
    const int t = rank + S * half + 2 * S * lane;
    if (t < M) {
      if (T::CONV && a.convert != 3) {
        const float most = __uint_as_float(ctl.most[t]);
        sx_own = most < INFINITY ? __fdiv_rn(most, 127.f) : __uint_as_float(0x7fffffffu);
      } else {
        sx_own = __ldcg(a.sx + t);
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (warp >= 4) {
    const uint32_t part = smem_u32(smem) + 4 * r;
    int at = 0;  // which of this warp's tokens
#pragma unroll 1
    for (int t0 = first; t0 < M; t0 += 2 * S * AT_ONCE, at += AT_ONCE) {
      float v[AT_ONCE][P];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
#pragma unroll
        for (int p = 0; p < P; ++p) v[j][p] = 0.f;
      uint32_t kept[3][AT_ONCE] = {};
#pragma unroll
      for (int i = 0; i < 3 && T::BACK == DHIDDEN; ++i) kept[i][0] = next[i].x, kept[i][1] = next[i].y, kept[i][2] = next[i].z, kept[i][3] = next[i].w;
      load_kept(t0 + 2 * S * AT_ONCE);
#pragma unroll 4
      for (int c = 0; c < S; ++c) {
        uint32_t from;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(part), "r"(c));
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
          const int t = min(t0 + apart * j, M - 1);
#pragma unroll
          for (int p = 0; p < P; ++p) v[j][p] += ld_cluster1(from + (p * NT + t) * (BM * 4));
        }
      }
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const int t = t0 + apart * j;
        if (t >= M) break;
        if (T::I8) {
          // (at most 64 tokens a warp, of which the second 32 come with one CTA to 128 tokens alone)
          const float sx = at + j < 32 ? __shfl_sync(0xffffffffu, sx_own, (at + j) & 31) : __ldcg(a.sx + t);
          v[j][0] *= sx * sw;
          if (T::GATED) v[j][P - 1] *= sx * sw1;
        }
        if (T::GATED) {
          const float g = v[j][0], u = v[j][P - 1], h = silu_mul(g, u);
          if (T::I8) {
            if (is) a.hf[static_cast<size_t>(t) * N + ch] = h;
            const unsigned most = __reduce_max_sync(0xffffffffu, is ? __float_as_uint(max_abs(0.f, h, 0.f)) : 0u);
            if (lane == 0) atomicMax(&ctl.hmost[t], most);
          } else {
            if (is) a.h[static_cast<size_t>(t) * N + ch] = static_cast<uint16_t>(pack_bf16x2(h, 0.f));
            if (a.saved) {
              // the words of two channels (pop_wide16.h): the even one's lane has the first and the last, the odd one's
              // the second
              const uint32_t gb = __float_as_uint(g), ub = __float_as_uint(u);
              const uint32_t gn = __shfl_xor_sync(0xffffffffu, gb, 1), un = __shfl_xor_sync(0xffffffffu, ub, 1);
              kept[0][j] = __byte_perm(gb, gn, 0x7632);
              kept[1][j] = __byte_perm(un, ub, 0x7632);
              kept[2][j] = __byte_perm(__byte_perm(gb, gn, 0x0051), __byte_perm(ub, un, 0x0051), 0x5410);
            }
          }
        } else if (T::BACK == DHIDDEN) {
          const float g = __uint_as_float(__byte_perm(kept[0][j], kept[2][j], lane & 1 ? 0x3255 : 0x1044));
          const float u = __uint_as_float(__byte_perm(kept[1][j], kept[2][j], lane & 1 ? 0x3277 : 0x1066));
          const float p = sigmoid(g), d = v[j][0];
          const size_t o = static_cast<size_t>(t) * N + ch;
          if (is) {
            a.h[o] = static_cast<uint16_t>(pack_bf16x2(d * u * (p * fmaf(g, 1.f - p, 1.f)), 0.f));
            a.h2[o] = static_cast<uint16_t>(pack_bf16x2(d * (g * p), 0.f));
          }
        } else if (is) {
          const size_t o = static_cast<size_t>(t) * a.ldy[0] + ch;
          if (a.out_f32)
            static_cast<float*>(a.y[0])[o] = v[j][0];
          else
            static_cast<uint16_t*>(a.y[0])[o] = static_cast<uint16_t>(pack_bf16x2(v[j][0], 0.f));
        }
      }
      if (T::GATED && !T::I8 && a.saved && is) {
        // (of a last few tokens also the words behind them, which 32 rows together have room for)
        uint4* k = reinterpret_cast<uint4*>(a.saved + (static_cast<size_t>(t0 >> 5) * (N >> 1) + (ch >> 1)) * 96 + (t0 & 31));
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if ((lane & 1) == (i & 1)) __stcg(k + 8 * i, make_uint4(kept[i][0], kept[i][1], kept[i][2], kept[i][3]));
      }
    }
    if (T::I8 && T::GATED) {
      if (half)  // the half's four warps
        asm volatile("bar.sync 4, 128;" ::: "memory");
      else
        asm volatile("bar.sync 3, 128;" ::: "memory");
      for (int i = 32 * q + lane; rank + S * (half + 2 * i) < M; i += 128) {
        const int t = rank + S * (half + 2 * i);
        a.amax[static_cast<size_t>(tile) * THIN16_MOST + t] = ctl.hmost[t];
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // nothing of this CTA is still used by another
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, T::TMEM_COLS);
  }
}

// The kernel's shared memory. Every one of them wants all of it for its SMs: otherwise they are set up for two CTAs of its own
// size, and the next kernel's wait for those to leave (64 rows by 2 x 5496 x 2048 and back 25 -> 20 us, 40 by 2 x 2736 x 1000 14.4 ->
// 13.3). The kernels that quantise rows do without: 24 rows of the latter in 8 bits, 16.1 us, took 0.6 more.
template <class T>
cudaError_t prepare() {
  static std::atomic<bool> known[64];
  const void* kernel = reinterpret_cast<const void*>(&k_thin16<T>);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = ensure_dyn_smem(kernel, T::SMEM);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && dev < 64) known[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <class T>
cudaError_t launch(WArgs a, cudaStream_t st) {
  const cudaError_t e = prepare<T>();
  if (e != cudaSuccess) return e;
  for (int i = 0; i < T::SEGMENTS && !T::CONV; ++i)
    if (!encode_map16(&a.map[2 * i], i ? a.rows2 : a.rows, a.k, a.m[0], static_cast<uint64_t>(a.ld_rows) * 2, BK, T::NT)) return cudaErrorInvalidValue;
  const int tiles = qceil(a.n[0], BM), S = thin16_split(T::I8, a.m[0], a.n[0], a.kb * T::SEGMENTS, a.num_sms);
  if (T::CONV && qceil(a.kb, S) > THIN16_KEPT) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(S), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * S);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = T::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_thin16<T>, a);
}

template <bool I8, bool GATED, Back BACK = FORWARD>
cudaError_t by_rows(const WArgs& a, cudaStream_t st) {
  if (I8 && a.convert) return launch<Thin<I8, GATED, 16, I8>>(a, st);
  if (a.m[0] <= 16) return launch<Thin<I8, GATED, 16, false, BACK>>(a, st);
  if (a.m[0] <= 32) return launch<Thin<I8, GATED, 32, false, BACK>>(a, st);
  return a.m[0] <= 64 ? launch<Thin<I8, GATED, 64, false, BACK>>(a, st) : launch<Thin<I8, GATED, 128, false, BACK>>(a, st);
}

// Clusters of S CTAs that the device holds at a time with a CTA on each SM; asked once per device. (Of 152 SMs 36 of 4, 23
// of 6, 15 of 7 or 8.)
int clusters_at_a_time(int S, int num_sms) {
  using T = Thin<false, false, 128>;
  static std::atomic<int> known[64][9];
  int dev = 0;
  if (S == 1) return num_sms;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][S].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(S), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / S * S);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = T::SMEM;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (prepare<T>() != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k_thin16<T>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = n > 0 ? n : -1;
    known[dev][S].store(n, std::memory_order_relaxed);
  }
  return n > 0 ? n : 0;
}

}  // namespace

// As many CTAs to a tile as have an SM each, in clusters of their number; a few clusters that have to wait for the others
// cost as much again (64 rows by 2 x 5496 x 2048 and back: 33 us in clusters of 7, 22 in clusters of 3). Two on an SM where each
// still has 16 k-blocks (one row by 2 x 11008 x 4096 and back: clusters of 3 47.9 us, of 1 53.8), or 6, where else only one
// would be at a tile and SMs idle (32 rows of 8 bits by 11008 x 2048: 11.1 with 3, 14.1 with 1; 128 rows by 11008 x 8192, one
// after the other: 39.5 and 48.7). No more than have four k-blocks or 16 tokens each: a larger cluster takes longer to
// meet than it saves (16 rows by 2 x 2736 x 1000, back and forth: 45 us with 8, 40 with 4; 64 rows by 2 x 1024 x 256, a block
// each: 33 with 4, 41 with 1).
int thin16_split(bool i8, int m, int n, int kb, int num_sms) {
  const int tiles = qceil(n, BM);
  int one = 1, two = 1;
  for (int S = 2; S <= 8; ++S) {
    const int held = clusters_at_a_time(S, num_sms);
    if (held >= tiles) one = S;
    if (tiles * S <= 2 * num_sms && 2 * held * 11 >= tiles * 10) two = S;  // (a tenth too many does no harm)
  }
  const bool pays = one == 1 ? kb / two >= 6 && (i8 || m <= 64) : kb / two >= 16 && m <= 64;  // (of more rows one fits on an SM)
  const int use = std::max(kb / 4, qceil(m, 16));
  return std::max(1, std::min({pays ? std::max(one, two) : one, use, kb}));
}

bool thin16_converts(int convert, int m, int n, int k, int num_sms) {
  if (m > 16) return false;
  const int kb = qceil(k, BK);
  const long long values = static_cast<long long>(m) * k;
  return qceil(kb, thin16_split(true, m, n, kb, num_sms)) <= THIN16_KEPT && (convert == 3 || values <= (convert == 1 ? 12288 : 45056));
}

cudaError_t launch_thin16(WKind kind, const WArgs& a, cudaStream_t st) {
  switch (kind) {
    case W_GATED: return by_rows<false, true>(a, st);
    case W_PLAIN: return by_rows<false, false>(a, st);
    case W_DGATED: return by_rows<false, false, DHIDDEN>(a, st);
    case W_DX: return by_rows<false, false, DROWS>(a, st);
    case W_I8: return by_rows<true, false>(a, st);
    case W_I8_GATED: return by_rows<true, true>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pop
