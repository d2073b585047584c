// Products of few rows (tokens) and a matrix in e4m3 with block scales: the matrix streams once.
//
// y[n][f] = sum over k-blocks b of s_x[n][b] s_w[f/128][b] * (q_x[n] . q_w[f])_b. The matrix is the M operand
// (128 outputs f per tile), the tokens the N operand (NT = 16, 32 or 64 per tile, as many as there are,
// rounded up to 16). A k-block is one tcgen05 product of 128 x N x 128 into a TMEM buffer of its own,
// which the epilogue adds to fp32 registers with the block's scales. Bound by the matrix's bytes, so the
// split is one that keeps every SM streaming to the end: all (tile, k-block) pairs in order are cut into
// one equal run per CTA. A tile that lies in several runs is summed from fp32 parts in the order of k by
// whichever of its CTAs comes last (a counter per tile; no CTA waits for another), so the bits do not
// depend on the order in which CTAs run.
//
// Warp 0: copies (one bulk copy per stage for the matrix, its image being what shared memory needs; 2 KB
// per 16 tokens; the tokens' scales). Warp 1: products. Warps 2..5: epilogue, TMEM lane quarter warp % 4.
// Every wait has a limit; a CTA that gives up records QERR_TIMEOUT, lets its copies and products finish,
// frees TMEM and returns.
#include "pop_qdevice.cuh"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int THREADS = 192;
constexpr uint32_t RING_BYTES = 200 * 1024;
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_STAGES = 16, MAX_BUFS = 8;

template <bool GATED, int NT>
struct Thin {
  static constexpr int P = GATED ? 2 : 1;
  static constexpr uint32_t W_BYTES = P * QTILE;
  static constexpr uint32_t X_BYTES = NT * QB;
  static constexpr uint32_t STAGE = (W_BYTES + X_BYTES + NT * 4 + 1023) / 1024 * 1024;
  static constexpr int STAGES = RING_BYTES / STAGE < MAX_STAGES ? RING_BYTES / STAGE : MAX_STAGES;
  static constexpr int BUFS = static_cast<int>(TMEM_COLS) / (P * NT) < MAX_BUFS ? static_cast<int>(TMEM_COLS) / (P * NT) : MAX_BUFS;
};

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t tfull[MAX_BUFS], tempty[MAX_BUFS];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int last;
  Groups groups;
  uint32_t amax[4][64];
};

// One run of k-blocks of a tile.
struct Seg {
  int tile, kb0, kb1;
  int e, t, n0, n;  // group, output tile, first token and number of tokens of the tile
  int row0;         // first row
};

template <int NT>
__device__ __forceinline__ Seg segment(const Groups& gr, int E, int KB, long long x, long long x1) {
  Seg s;
  s.tile = static_cast<int>(x / KB);
  s.kb0 = static_cast<int>(x - static_cast<long long>(s.tile) * KB);
  s.kb1 = static_cast<int>(min(static_cast<long long>(KB), s.kb0 + (x1 - x)));
  s.e = gr.of(E, s.tile);
  const int cnt = gr.count[s.e];
  const int tts = qceil(cnt, NT);
  const int local = s.tile - gr.tile0[s.e];
  s.t = local / tts;  // the token tiles of one output tile side by side: the matrix tile is in L2 for the others
  s.n0 = (local - s.t * tts) * NT;
  s.n = min(NT, cnt - s.n0);
  s.row0 = gr.run0[s.e] * 16 + s.n0;
  return s;
}

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <bool GATED, int NT>
__global__ void __launch_bounds__(THREADS, 1) k_qgemm_thin(const __grid_constant__ QGemmArgs a) {
  using C = Thin<GATED, NT>;
  constexpr int P = C::P;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = qceil(a.K, QB), NTILES = qceil(a.N, QB);
  volatile int* abort_flag = &ctl.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1 + 4);  // the products and the epilogue's four warps (scales)
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(&ctl.tfull[b], 1);
      mbar_init(&ctl.tempty[b], 4);
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
  const int tiles = ctl.groups.fill(a, NT, NTILES);
  const long long work = static_cast<long long>(tiles) * KB;
  const long long G = min(static_cast<long long>(gridDim.x), work);  // CTAs that have a unit
  const bool on = static_cast<long long>(blockIdx.x) < G;
  const long long x0 = on ? work * blockIdx.x / G : 0, x1 = on ? work * (blockIdx.x + 1) / G : 0;

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
      for (long long x = x0; x < x1 && ok;) {
        const Seg g = segment<NT>(ctl.groups, a.E, KB, x, x1);
        const int runs = qceil(g.n, 16);
        const uint8_t* w = a.w + g.e * a.w_stride + static_cast<size_t>(g.t) * KB * C::W_BYTES;
        const uint8_t* xr = a.act + static_cast<size_t>(g.row0 / 16) * KB * 2048;
        const uint32_t bytes = C::W_BYTES + runs * (2048 + 64);
        for (int kb = g.kb0; kb < g.kb1; ++kb, ++issued) {
          const int s = issued % C::STAGES;
          if (!mbar_wait(&ctl.empty[s], ((issued / C::STAGES) & 1u) ^ 1u, Q_WAIT_NS, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::STAGE;
          mbar_arrive_expect_tx(&ctl.full[s], bytes);
          bulk_load(st, w + static_cast<size_t>(kb) * C::W_BYTES, C::W_BYTES, &ctl.full[s]);
          for (int r = 0; r < runs; ++r)
            bulk_load(st + C::W_BYTES + r * 2048, xr + (static_cast<size_t>(r) * KB + kb) * 2048, 2048, &ctl.full[s]);
          bulk_load(st + C::W_BYTES + C::X_BYTES, a.act_s + static_cast<size_t>(kb) * a.rows + g.row0, runs * 64,
                    &ctl.full[s]);
        }
        x += g.kb1 - g.kb0;
      }
      // no copy of this CTA may be in flight when it exits
      const uint32_t lo = issued > C::STAGES ? issued - C::STAGES : 0;
      for (uint32_t i = lo; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.full[i % C::STAGES], (i / C::STAGES) & 1u, Q_DRAIN_NS, &never)) fail();
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------- products (one thread)
      uint32_t it = 0;
      bool ok = true;
      for (long long x = x0; x < x1 && ok;) {
        const Seg g = segment<NT>(ctl.groups, a.E, KB, x, x1);
        const uint32_t idesc = idesc_e4m3_f32(128, qceil(g.n, 16) * 16);
        for (int kb = g.kb0; kb < g.kb1; ++kb, ++it) {
          const int s = it % C::STAGES, b = it % C::BUFS;
          if (!mbar_wait(&ctl.full[s], (it / C::STAGES) & 1u, Q_WAIT_NS, abort_flag) ||
              !mbar_wait(&ctl.tempty[b], ((it / C::BUFS) & 1u) ^ 1u, Q_WAIT_NS, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * C::STAGE);
          const uint32_t d = tmem_base + static_cast<uint32_t>(b * P * NT);
          umma_block(d, st, st + C::W_BYTES, idesc);
          if (GATED) umma_block(d + NT, st + QTILE, st + C::W_BYTES, idesc);
          umma_commit(&ctl.empty[s]);
          umma_commit(&ctl.tfull[b]);
        }
        x += g.kb1 - g.kb0;
      }
      umma_commit(&ctl.drain);
      volatile int never = 0;
      if (!mbar_wait(&ctl.drain, 0, Q_DRAIN_NS, &never)) fail();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..5)
    const int q = warp & 3;
    const int f = 32 * q + lane;  // output of the tile
    const int et = threadIdx.x - 64;
    uint32_t it = 0;
    for (long long x = x0; x < x1;) {
      const Seg g = segment<NT>(ctl.groups, a.E, KB, x, x1);
      const float* ws = a.ws + g.e * a.ws_stride + static_cast<size_t>(g.t) * scale_stride(KB, P);
      float acc[P][NT];
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[p][n] = 0.f;
      float sw = 0.f;  // lane i: the matrix's scale number 32 j + i of this run
      bool ok = true;
      for (int kb = g.kb0; kb < g.kb1; ++kb, ++it) {
        const int i = (kb - g.kb0) * P;
        if ((i & 31) == 0) sw = i + lane < (g.kb1 - g.kb0) * P ? __ldg(ws + static_cast<size_t>(g.kb0) * P + i + lane) : 0.f;
        const int s = it % C::STAGES, b = it % C::BUFS;
        ok = mbar_wait(&ctl.full[s], (it / C::STAGES) & 1u, Q_WAIT_NS, abort_flag) &&
             mbar_wait(&ctl.tfull[b], (it / C::BUFS) & 1u, Q_WAIT_NS, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float4* sx = reinterpret_cast<const float4*>(smem + s * C::STAGE + C::W_BYTES + C::X_BYTES);
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * P * NT);
        const float s0 = __shfl_sync(0xffffffffu, sw, i & 31), s1 = __shfl_sync(0xffffffffu, sw, (i + P - 1) & 31);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          if (c >= g.n) break;
          uint32_t d0[16], d1[16];
          tmem_ld16(taddr + c, d0);
          if (GATED) tmem_ld16(taddr + NT + c, d1);
          tmem_wait16(d0);
          if (GATED) tmem_wait16(d1);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 v = sx[(c + j) >> 2];
            const float vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              acc[0][c + j + r] = fmaf(s0 * vs[r], __uint_as_float(d0[j + r]), acc[0][c + j + r]);
              if (GATED) acc[P - 1][c + j + r] = fmaf(s1 * vs[r], __uint_as_float(d1[j + r]), acc[P - 1][c + j + r]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.tempty[b]);
          mbar_arrive(&ctl.empty[s]);
        }
      }
      if (!ok && lane == 0) fail();
      if (epi_any<128>(!ok)) break;  // all four warps go on, or none
      x += g.kb1 - g.kb0;
      if (g.kb1 - g.kb0 < KB) {
        // a part of the tile. Slot 0 of this CTA holds one that starts within its tile, slot 1 one that
        // starts it: a run has at most one of each.
        const size_t slot_floats = static_cast<size_t>(P) * NT * 128;
        float* mine = a.parts + (2 * static_cast<size_t>(blockIdx.x) + (g.kb0 == 0 ? 1 : 0)) * slot_floats + f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n < g.n) __stcg(mine + (p * NT + n) * 128, acc[p][n]);
        const long long first = static_cast<long long>(g.tile) * KB, last = first + KB - 1;
        // CTA c holds [work c / G, work (c + 1) / G): the one of unit x is ((x + 1) G - 1) / work
        const int c0 = static_cast<int>(((first + 1) * G - 1) / work), c1 = static_cast<int>(((last + 1) * G - 1) / work);
        __threadfence();
        epi_sync();
        if (et == 0) ctl.last = atomicAdd(a.done + g.tile, 1u) == static_cast<unsigned>(c1 - c0) ? 1 : 0;
        epi_sync();
        const bool mine_last = ctl.last != 0;
        epi_sync();  // ctl.last is free again
        if (!mine_last) continue;
        __threadfence();
        if (et == 0) a.done[g.tile] = 0;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[p][n] = 0.f;
        for (int c = c0; c <= c1; ++c) {
          const float* p0 = a.parts + (2 * static_cast<size_t>(c) + (work * c / G <= first ? 1 : 0)) * slot_floats + f;
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n < g.n) acc[p][n] += __ldcg(p0 + (p * NT + n) * 128);
        }
      }
      if (!GATED) {
        const int col = g.t * QB + f;
        if (col < a.N) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n < g.n) {
              const size_t o = static_cast<size_t>(g.row0 + n) * a.ldy + col;
              if (a.out_f32)
                static_cast<float*>(a.y)[o] = acc[0][n];
              else
                static_cast<__nv_bfloat16*>(a.y)[o] = __float2bfloat16_rn(acc[0][n]);
            }
          }
        }
      } else {
        // the tile's 128 channels are one block of the next product's rows
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n < g.n) {
            acc[0][n] = silu_mul(acc[0][n], acc[P - 1][n]);
            const uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits(acc[0][n]));
            if (lane == 0) ctl.amax[q][n] = m;
          }
        }
        epi_sync();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n < g.n) {
            const uint32_t m = max(max(max(ctl.amax[0][n], ctl.amax[1][n]), max(ctl.amax[2][n], ctl.amax[3][n])), AMAX_MIN_BITS);
            const float am = __uint_as_float(m);
            const bool huge = q_huge(am);
            const float v = q_ratio(acc[0][n], am, q_recip(am, huge), huge);
            const int r = g.row0 + n;
            a.h[(static_cast<size_t>(r / 16) * NTILES + g.t) * 2048 + image_at(r % 16, f)] =
                static_cast<uint8_t>(e4m3x2(v, 0.f));
            if (f == 0) a.h_s[static_cast<size_t>(g.t) * a.rows + r] = __fdiv_rn(am, 448.f);
          }
        }
        epi_sync();  // ctl.amax is free again
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

template <bool GATED, int NT>
cudaError_t launch(const QGemmArgs& a, cudaStream_t st) {
  using C = Thin<GATED, NT>;
  const size_t smem = C::STAGES * C::STAGE + 1024;
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(&k_qgemm_thin<GATED, NT>), smem);
  if (e != cudaSuccess) return e;
  return launch_q(k_qgemm_thin<GATED, NT>, dim3(a.num_sms), THREADS, smem, st, a);
}

}  // namespace

// Two slots per CTA of the widest kind of tile.
size_t qgemm_thin_parts(int num_sms, bool gated) { return static_cast<size_t>(2) * num_sms * 128 * 64 * (gated ? 2 : 1); }

cudaError_t launch_qgemm_thin(const QGemmArgs& a, bool gated, int max_rows, cudaStream_t st) {
  const int nt = max_rows <= 16 ? 16 : max_rows <= 32 ? 32 : 64;
  if (gated) return nt == 16 ? launch<true, 16>(a, st) : nt == 32 ? launch<true, 32>(a, st) : launch<true, 64>(a, st);
  return nt == 16 ? launch<false, 16>(a, st) : nt == 32 ? launch<false, 32>(a, st) : launch<false, 64>(a, st);
}

}  // namespace pop
