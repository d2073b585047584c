// Products of many rows (tokens) and a matrix in e4m3 with block scales, on 128 x 256 tiles.
//
// Rows are the M operand (128 per tile), the matrix the N operand: 256 outputs, or the gate and the up
// rows of 128 channels. A block of 128 in k has scales of its own, so its product cannot be added to the
// next one's in tensor memory: each k-block is one tcgen05 product of 128 x 256 x 128 into one of two
// TMEM buffers, which eight epilogue warps add to fp32 registers, times the row's scale (one per thread: a
// thread has one row) and the matrix's (one per 128 columns), while the tensor core fills the other.
// A k-block takes the tensor core 512 cycles; reading 256 columns of TMEM and 128 x 256 fused
// multiply-adds (two per instruction) about 300, so the products are what bounds it.
//
// Persistent, one CTA per SM. Warp 0: copies (operand images: bulk copies of 16 KB). Warp 1: products.
// Warps 2..9: epilogue, TMEM lane quarter warp % 4, two warps to a quarter that share its columns. Every wait
// has a limit; a CTA that gives up records QERR_TIMEOUT, lets its copies and products finish, frees TMEM
// and returns.
#include "pop_qdevice.cuh"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int THREADS = 320;
constexpr int BM = 128;
constexpr int STAGES = 4;
constexpr uint32_t A_BYTES = QTILE, B_BYTES = 2 * QTILE, STAGE = A_BYTES + B_BYTES;
constexpr uint32_t TMEM_COLS = 512;

struct Ctl {
  uint64_t full[STAGES], empty[STAGES];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int tile0[POP_QMOE_MAX_EXPERTS + 1];
  uint32_t amax[2][2][BM];  // gated: [tile parity][column half][row]
};

struct Tile {
  int e, n, m0, rows;  // group, tile of the matrix, first row within the group, rows of this tile
  int row0;            // first row
};

__device__ __forceinline__ Tile tile_at(const QGemmArgs& a, const int* tile0, int per, int tile) {
  Tile t;
  t.e = group_of(tile0, a.E, tile);
  const int cnt = a.counts ? __ldcg(a.counts + t.e) : a.M;
  const int mts = qceil(cnt, BM);
  const int local = tile - tile0[t.e];
  t.n = local / mts;  // the row tiles of one matrix tile side by side: it is in L2 for all of them
  t.m0 = (local - t.n * mts) * BM;
  t.rows = min(BM, cnt - t.m0);
  t.row0 = (a.run0 ? __ldcg(a.run0 + t.e) : 0) * BM + t.m0;
  return t;
}

template <bool GATED>
__global__ void __launch_bounds__(THREADS, 1) k_qgemm_wide(const __grid_constant__ QGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = qceil(a.K, QB), NT = qceil(a.N, QB);
  const int per = GATED ? NT : qceil(NT, 2);  // tiles of the matrix
  volatile int* abort_flag = &ctl.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.tfull[b], 1);
      mbar_init(&ctl.tempty[b], 8);
    }
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base;
  pdl_wait();  // the rows, the groups, and what an earlier call's kernels still use
  pdl_trigger();
  const int tiles = group_tiles(a, BM, per, ctl.tile0);

  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      atomicOr(a.err, QERR_TIMEOUT);
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- copies (one thread)
      uint32_t issued = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const Tile t = tile_at(a, ctl.tile0, per, tile);
        const uint8_t* xr = a.act + static_cast<size_t>(t.row0 / BM) * KB * A_BYTES;
        // gated: [tile][k-block][gate | up]; else tiles 2 n and 2 n + 1 (which may lie past the last)
        const uint8_t* w = a.w + t.e * a.w_stride + static_cast<size_t>(t.n) * KB * B_BYTES;
        const bool both = GATED || 2 * t.n + 1 < NT;
        for (int kb = 0; kb < KB; ++kb, ++issued) {
          const int s = issued % STAGES;
          if (!mbar_wait_bounded(&ctl.empty[s], ((issued / STAGES) & 1u) ^ 1u, Q_WAIT_NS, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = smem + s * STAGE;
          mbar_arrive_expect_tx(&ctl.full[s], A_BYTES + (both ? B_BYTES : QTILE));
          bulk_load(st, xr + static_cast<size_t>(kb) * A_BYTES, A_BYTES, &ctl.full[s]);
          if (GATED) {
            bulk_load(st + A_BYTES, w + static_cast<size_t>(kb) * B_BYTES, B_BYTES, &ctl.full[s]);
          } else {
            bulk_load(st + A_BYTES, w + static_cast<size_t>(kb) * QTILE, QTILE, &ctl.full[s]);
            if (both) bulk_load(st + A_BYTES + QTILE, w + static_cast<size_t>(KB + kb) * QTILE, QTILE, &ctl.full[s]);
          }
        }
      }
      // no copy of this CTA may be in flight when it exits
      const uint32_t lo = issued > STAGES ? issued - STAGES : 0;
      for (uint32_t i = lo; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait_bounded(&ctl.full[i % STAGES], (i / STAGES) & 1u, Q_DRAIN_NS, &never)) fail();
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------- products (one thread)
      constexpr uint32_t IDESC = idesc_e4m3_f32(BM, 256);
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int s = it % STAGES, b = it & 1;
          if (!mbar_wait_bounded(&ctl.full[s], (it / STAGES) & 1u, Q_WAIT_NS, abort_flag) ||
              !mbar_wait_bounded(&ctl.tempty[b], ((it >> 1) & 1u) ^ 1u, Q_WAIT_NS, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * STAGE);
          umma_block(tmem_base + static_cast<uint32_t>(b * 256), st, st + A_BYTES, IDESC);
          umma_commit(&ctl.empty[s]);
          umma_commit(&ctl.tfull[b]);
        }
      }
      umma_commit(&ctl.drain);
      volatile int never = 0;
      if (!mbar_wait_bounded(&ctl.drain, 0, Q_DRAIN_NS, &never)) fail();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int r = 32 * q + lane;  // row of the tile
    // this thread's columns: two runs of 64. Gated: gate and up of channels [64 half, 64 half + 64)
    const uint32_t col0 = GATED ? 64u * half : 128u * half;
    const uint32_t col1 = GATED ? 128u + 64u * half : 128u * half + 64u;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    uint32_t it = 0;
    int parity = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, parity ^= 1) {
      const Tile t = tile_at(a, ctl.tile0, per, tile);
      const float* xs = a.act_s + t.row0 + r;
      // scales of this thread's columns, k-block kb: ws[kb * step] (and ws[kb * step + 1] for up)
      const int wt = GATED ? t.n : min(2 * t.n + half, NT - 1);
      constexpr int STEP = GATED ? 2 : 1;
      const float* ws = a.ws + t.e * a.ws_stride + static_cast<size_t>(wt) * KB * STEP;
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      float sw = 0.f;                                                       // lane i: scale 32 j + i
      float sx0 = __ldcg(xs), sx1 = KB > 1 ? __ldcg(xs + a.rows) : 0.f;  // two k-blocks ahead
      for (int kb = 0; kb < KB; ++kb, ++it) {
        const int i = kb * STEP;
        if ((i & 31) == 0) sw = i + lane < KB * STEP ? __ldg(ws + i + lane) : 0.f;
        const float sx = sx0;
        sx0 = sx1;
        if (kb + 2 < KB) sx1 = __ldcg(xs + static_cast<size_t>(kb + 2) * a.rows);
        const float f0 = sx * __shfl_sync(0xffffffffu, sw, i & 31);
        const float f1 = GATED ? sx * __shfl_sync(0xffffffffu, sw, (i + 1) & 31) : f0;
        const int b = it & 1;
        ok = mbar_wait_bounded(&ctl.tfull[b], (it >> 1) & 1u, Q_WAIT_NS, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = lane_base + static_cast<uint32_t>(b * 256);
        uint32_t d0[32], d1[32];
        tmem_ld32(taddr + col0, d0);
        tmem_wait32(d0);
        tmem_ld32(taddr + col0 + 32, d1);
#pragma unroll
        for (int j = 0; j < 16; ++j) fma2(acc[j], __uint_as_float(d0[2 * j]), __uint_as_float(d0[2 * j + 1]), f0);
        tmem_wait32(d1);
        tmem_ld32(taddr + col1, d0);
#pragma unroll
        for (int j = 0; j < 16; ++j) fma2(acc[16 + j], __uint_as_float(d1[2 * j]), __uint_as_float(d1[2 * j + 1]), f0);
        tmem_wait32(d0);
        tmem_ld32(taddr + col1 + 32, d1);
#pragma unroll
        for (int j = 0; j < 16; ++j) fma2(acc[32 + j], __uint_as_float(d0[2 * j]), __uint_as_float(d0[2 * j + 1]), f1);
        tmem_wait32(d1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.tempty[b]);
#pragma unroll
        for (int j = 0; j < 16; ++j) fma2(acc[48 + j], __uint_as_float(d1[2 * j]), __uint_as_float(d1[2 * j + 1]), f1);
      }
      if (!ok && lane == 0) fail();
      if (!GATED && !ok) break;
      const bool valid = r < t.rows;
      const int row = t.row0 + r;
      if (GATED) {
        uint32_t m = AMAX_MIN_BITS;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          acc[j].x = silu_mul(acc[j].x, acc[32 + j].x);
          acc[j].y = silu_mul(acc[j].y, acc[32 + j].y);
          m = max(m, max(abs_bits(acc[j].x), abs_bits(acc[j].y)));
        }
        // the block of 128 channels is shared with the thread of the other half
        ctl.amax[parity][half][r] = m;
        if (epi_any<256>(!ok)) break;  // all eight warps go on, or none
        m = max(m, ctl.amax[parity][half ^ 1][r]);
        if (valid) {
          const float am = __uint_as_float(m);
          uint8_t* hp = a.h + (static_cast<size_t>(row / BM) * NT + t.n) * A_BYTES;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(hp + image_at(r, 64 * half + 16 * c)) =
                e4m3x16(reinterpret_cast<const float*>(acc) + 16 * c, am);
          if (half == 0) a.h_s[static_cast<size_t>(t.n) * a.rows + row] = __fdiv_rn(am, 448.f);
        }
      } else if (valid) {
        const int col = 256 * t.n + 128 * half;
        const int cols = min(128, a.N - col);
        const size_t o = static_cast<size_t>(row) * a.ldy + col;
        if (a.out_f32) {
          float* y = static_cast<float*>(a.y) + o;
          if (cols == 128 && (reinterpret_cast<uintptr_t>(y) & 15) == 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              reinterpret_cast<float4*>(y)[j] = make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
          } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              if (2 * j < cols) y[2 * j] = acc[j].x;
              if (2 * j + 1 < cols) y[2 * j + 1] = acc[j].y;
            }
          }
        } else {
          uint16_t* y = static_cast<uint16_t*>(a.y) + o;
          if (cols == 128 && (reinterpret_cast<uintptr_t>(y) & 15) == 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              reinterpret_cast<uint4*>(y)[j] =
                  make_uint4(pack_bf16x2(acc[4 * j].x, acc[4 * j].y), pack_bf16x2(acc[4 * j + 1].x, acc[4 * j + 1].y),
                             pack_bf16x2(acc[4 * j + 2].x, acc[4 * j + 2].y), pack_bf16x2(acc[4 * j + 3].x, acc[4 * j + 3].y));
          } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              const uint32_t v = pack_bf16x2(acc[j].x, acc[j].y);
              if (2 * j < cols) y[2 * j] = static_cast<uint16_t>(v);
              if (2 * j + 1 < cols) y[2 * j + 1] = static_cast<uint16_t>(v >> 16);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace

cudaError_t launch_qgemm_wide(const QGemmArgs& a, bool gated, cudaStream_t st) {
  const size_t smem = STAGES * STAGE + 1024;
  const void* k = gated ? reinterpret_cast<const void*>(&k_qgemm_wide<true>) : reinterpret_cast<const void*>(&k_qgemm_wide<false>);
  const cudaError_t e = ensure_dyn_smem(k, smem + sizeof(Ctl));
  if (e != cudaSuccess) return e;
  return gated ? launch_q(k_qgemm_wide<true>, dim3(a.num_sms), THREADS, smem, st, a)
               : launch_q(k_qgemm_wide<false>, dim3(a.num_sms), THREADS, smem, st, a);
}

}  // namespace pop
