// Products of many rows (tokens) and a matrix in e4m3 with block scales, on 128 x 256 tiles.
//
// Rows are the M operand, the matrix the N operand: 256 outputs, or the gate and the up rows of 128
// channels. Two CTAs of a cluster work as a pair on 256 rows by 256 outputs (cta_group::2): each brings its own
// 128 rows and half of the matrix tile, 32 KB a k-block instead of the 48 KB of a CTA alone, which at the 512
// cycles of a k-block's product would be 94 bytes a cycle and SM (bulk copies alone brought 78 to 105 from L2).
// Measured: a k-block takes 640 to 700 cycles, 4001 rows by 28672 x 8192 611 us alone (3.08 PFLOP/s) and 711 in a loop,
// which the power limit holds at 1.6 GHz; CTAs alone took 1068. Four fifths of the operands' bytes come from L2 (4096
// tokens through 2 of 8 experts of 4096 x 14336, gate and up: 0.99 GB from memory; tensor cores busy 67 %).
//
// A block of 128 in k has scales of its own, so its product cannot be added to the next one's in tensor
// memory: the epilogue adds each k-block's product to fp32 registers, times the row's scale (a thread has one
// row) and the matrix's. Tensor memory holds two k-blocks. Each is in halves, of 64 rows of either CTA's part
// of the matrix tile; a half has its own four epilogue warps, its own issuing thread and its own barriers, so
// that one is read while the other is being filled and half the latency from product to epilogue and back
// (some 600 cycles) is out of the way.
//
// The tiles go round the pairs, neighbours at the same time, so that what is in L2 serves many. Those that are left
// for a last round that would not be full are cut into one equal run of k-blocks per pair; a tile in several runs is
// summed from fp32 parts in the order of k by whichever of its pairs comes last (a counter per tile and CTA).
//
// Persistent, one CTA per SM. Warp 0: copies (operand images: bulk copies of 16 KB). Warps 1 and 3: of the first
// CTA the products of both CTAs, a half each; warp 1 of the second the news that its operands have landed.
// Warp 2: scales. Warps 4..11: epilogue, TMEM lane quarter warp % 4. Every wait has a limit; a CTA that gives
// up records QERR_TIMEOUT, lets its copies and products finish, frees TMEM and returns.
#include "pop_qdevice.cuh"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int THREADS = 384;
// Registers a thread: the launch has 168 (65,536 / 384, in eights); the epilogue's two warpgroups hold 128
// sums and up to 64 columns on their way, which at 168 spilled seven words a k-block.
constexpr int REGS = 168, REGS_COPY = 88, REGS_EPI = 208;
static_assert(REGS_COPY + 2 * REGS_EPI <= 3 * REGS, "the shares come out of the launch's registers");
constexpr int BM = 128;
constexpr int STAGES = 5;
constexpr uint32_t A_BYTES = QTILE, B_BYTES = QTILE, STAGE = A_BYTES + B_BYTES;
constexpr uint32_t TMEM_COLS = 512;

// Scales of eight k-blocks: the rows', and the matrix's of either half of the columns (gated: the gate's and the
// up's of each k-block, in turn).
constexpr int SB = 8, SRING = 4;
struct alignas(16) Scales {
  float x[SB][BM];
  float w[2 * SB];
};

// Plain: 128 bytes of 32 rows on their way out, of each epilogue warp, behind the ring.
constexpr uint32_t OUT_BYTES = 8 * 32 * 128;

struct Ctl {
  Scales scales[SRING];
  uint64_t sfull[SRING], sempty[SRING];
  uint64_t full[STAGES], empty[STAGES];
  uint64_t tfull[2][2], tempty[2][2];  // [half][buffer]
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int last;
  Groups groups;
  float amax[2][2][BM];  // gated: [tile parity][column half][row]
};

struct Tile {
  int e, n, m0, rows;  // group, tile of the matrix, first row within the group, rows of this CTA (may be none)
  int row0;            // first row; one that exists if there are none
};

__device__ __forceinline__ Tile tile_at(const Groups& g, int E, int tile, int rank) {
  Tile t;
  t.e = g.of(E, tile);
  const int cnt = g.count[t.e];
  const int mts = qceil(cnt, 2 * BM);
  const int local = tile - g.tile0[t.e];
  t.n = local / mts;  // the row tiles of one matrix tile side by side: it is in L2 for all of them
  t.m0 = (local - t.n * mts) * 2 * BM;
  t.rows = min(BM, cnt - t.m0 - rank * BM);
  if (t.rows > 0) t.m0 += rank * BM;
  t.row0 = g.run0[t.e] * BM + t.m0;
  return t;
}

// The tiles of one pair, in order, each with its k-blocks: whole ones, then its run of the last round's.
constexpr int SPLIT = 4;  // k-blocks of a run's unit: the scales of four begin on 16 bytes
struct Walk {
  int tile, kb0, kb1;
  // the split tiles: `units` units in all, over `sharers` pairs
  int first_split, units, sharers, KG;

  __device__ __forceinline__ Walk(int tiles, int pair, int pairs, int KB) : KB_(KB), pairs_(pairs) {
    const int rest = tiles % pairs;
    KG = qceil(KB, SPLIT);
    // A round takes KB k-blocks of 0.35 us or so. The split one takes KB * rest / pairs of them and some 20 us for the
    // parts, 128 KB of them per run and CTA written and read again (96 rows by 8192 x 28672: 32 tiles of 224 k-blocks, 83
    // us whole, 64 split; by 28672 x 8192, 36 tiles of 64 left: 59 whole, 65 split).
    const bool split = rest > 0 && KB * (pairs - rest) >= 72 * pairs;
    first_split = split ? tiles - rest : tiles;
    units = split ? rest * KG : 0;
    sharers = min(pairs, units);
    u_ = start(pair);
    u1_ = pair < sharers ? start(pair + 1) : u_;
    tile = pair - pairs;
    next();
  }
  __device__ __forceinline__ int start(int p) const {
    return p < sharers ? static_cast<int>(static_cast<long long>(units) * p / sharers) : units;
  }
  // the pair that holds unit u
  __device__ __forceinline__ int holder(int u) const {
    return static_cast<int>(((static_cast<long long>(u) + 1) * sharers - 1) / units);
  }
  __device__ __forceinline__ bool more() const { return kb1 > kb0; }
  __device__ __forceinline__ void next() {
    tile += pairs_;
    kb0 = 0;
    kb1 = KB_;
    if (tile < first_split) return;
    const int t = units > 0 ? u_ / KG : 0, k = u_ - t * KG;
    const int n = min(KG - k, u1_ - u_);
    tile = first_split + t - pairs_;
    kb0 = k * SPLIT;
    kb1 = n > 0 ? min(KB_, (k + n) * SPLIT) : kb0;
    tile += pairs_;
    u_ += n;
    at_tail_ = true;
  }
  __device__ __forceinline__ void advance() {
    if (at_tail_) tile = first_split - pairs_;  // the units say where to go on
    next();
  }

 private:
  int KB_, pairs_, u_, u1_;
  bool at_tail_ = false;
};

template <bool GATED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) k_qgemm_wide(const __grid_constant__ QGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int KB = qceil(a.K, QB), NT = qceil(a.N, QB);
  const int per = GATED ? NT : qceil(NT, 2);  // tiles of the matrix
  volatile int* abort_flag = &ctl.abort_flag;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl.full[s], rank == 0 ? 2 : 1);  // the first CTA's: its own operands, and word of the second's
      mbar_init(&ctl.empty[s], 2);
    }
    for (int g = 0; g < SRING; ++g) {
      mbar_init(&ctl.sfull[g], 1);
      mbar_init(&ctl.sempty[g], 8);
    }
    for (int b = 0; b < 2; ++b) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&ctl.tfull[h][b], 1);
        mbar_init(&ctl.tempty[h][b], 8);  // the first CTA's: the half's epilogue warps of both
      }
      mbar_init(&ctl.drain[b], 1);
    }
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl.tmem_base, TMEM_COLS);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base;
  // The groups' numbers, or the experts that they are counted from, are two kernels back or more: the kernel before this
  // waited for them before it let this one start (as this one does: pdl_trigger comes after a pdl_wait).
  const int tiles = ctl.groups.fill<false>(a, 2 * BM, per);

  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      atomicOr(a.err, QERR_TIMEOUT);
    }
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_COPY));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- copies (one thread)
      // (lean loops here and below: one thread's instructions follow one another at its latencies, and divisions
      // and 64-bit products once made these take longer than the products)
      uint32_t issued = 0, s = 0, phase = 1;
      bool ok = true, waited = false;
      for (Walk v(tiles, pair, pairs, KB); v.more() && ok; v.advance()) {
        const Tile t = tile_at(ctl.groups, a.E, v.tile, rank);
        const uint8_t* xr = a.act + (static_cast<size_t>(t.row0 / BM) * KB + v.kb0) * A_BYTES;
        // this CTA's half of the matrix tile. Gated: [tile][k-block][gate | up]; else tile 2 n + rank, or the
        // last one again
        const uint8_t* w = a.w + t.e * a.w_stride +
                           (GATED ? ((static_cast<size_t>(t.n) * KB + v.kb0) * 2 + rank)
                                  : static_cast<size_t>(min(2 * t.n + rank, NT - 1)) * KB + v.kb0) * QTILE;
        // A CTA without rows multiplies what its stages hold, and nothing reads the products (8 x (2 x 14336 x 4096), 80 to
        // 128 rows: 168 us, 175 with a copy of rows that are not used).
        const uint32_t xbytes = t.rows > 0 ? A_BYTES : 0;
        int kb = v.kb0;
        if (!waited) {
          // the matrix does not depend on the kernel before: the first stages' part of it goes out ahead of the rows
          const int ahead = min(STAGES, v.kb1 - v.kb0);
          for (int i = 0; i < ahead; ++i) {
            mbar_arrive_expect_tx(&ctl.full[i], xbytes + B_BYTES);
            bulk_load(smem + i * STAGE + A_BYTES, w + static_cast<size_t>(i) * (GATED ? 2 * QTILE : QTILE), QTILE, &ctl.full[i]);
          }
          pdl_wait();
          waited = true;
          for (int i = 0; i < ahead && xbytes; ++i) bulk_load(smem + i * STAGE, xr + static_cast<size_t>(i) * A_BYTES, A_BYTES, &ctl.full[i]);
          kb += ahead;
          xr += static_cast<size_t>(ahead) * A_BYTES;
          w += static_cast<size_t>(ahead) * (GATED ? 2 * QTILE : QTILE);
          issued = ahead;
          s = ahead;
          if (s == STAGES) s = 0, phase ^= 1;
        }
        for (; kb < v.kb1; ++kb) {
          if (!mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = smem + s * STAGE;
          mbar_arrive_expect_tx(&ctl.full[s], xbytes + B_BYTES);
          if (xbytes) bulk_load(st, xr, A_BYTES, &ctl.full[s]);
          bulk_load(st + A_BYTES, w, QTILE, &ctl.full[s]);
          xr += A_BYTES;
          w += GATED ? 2 * QTILE : QTILE;
          ++issued;
          if (++s == STAGES) s = 0, phase ^= 1;
        }
      }
      // no copy of this CTA may be in flight when it exits. (The first CTA's barriers also wait for word of the second,
      // which does not come if that one has given up; the copies have had their time when one such wait has run out.)
      const uint32_t lo = issued > STAGES ? issued - STAGES : 0;
      for (uint32_t i = lo; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.full[i % STAGES], (i / STAGES) & 1u, Q_DRAIN, &never)) {
          fail();
          break;
        }
      }
    }
    if (warp & 1) {
      uint32_t total = 0;  // k-blocks
      for (Walk v(tiles, pair, pairs, KB); v.more(); v.advance()) total += v.kb1 - v.kb0;
      const bool leader = elect_one();
      uint32_t s = 0, phase = 0;
      if (rank == 0) {
        // -------------------------------------------------------- products (a warp for either half)
        constexpr uint32_t IDESC = idesc_e4m3_f32(2 * BM, 128);
        const uint32_t h = static_cast<uint32_t>(warp >> 1);
        const uint32_t a0 = desc_lo(smem_u32(smem)), b0 = desc_lo(smem_u32(smem) + A_BYTES + h * (QTILE / 2));
        for (uint32_t it = 0; it < total; ++it) {
          const uint32_t b = it & 1u;
          if (!mbar_wait(&ctl.full[s], phase, a.wait, abort_flag) ||
              !mbar_wait(&ctl.tempty[h][b], ((it >> 1) & 1u) ^ 1u, a.wait, abort_flag)) {
            if (leader) fail();
            break;
          }
          tc_fence_after();
          if (leader) {
            umma_block_pair(tmem_base + b * 256u + h * 128u, a0 + s * (STAGE >> 4), b0 + s * (STAGE >> 4), IDESC);
            umma_commit_pair(&ctl.tfull[h][b]);
            umma_commit_pair(&ctl.empty[s]);
          }
          __syncwarp();
          if (++s == STAGES) s = 0, phase ^= 1;
        }
        if (leader) umma_commit_pair(&ctl.drain[h]);
        volatile int never = 0;
        if (!mbar_wait(&ctl.drain[h], 0, Q_DRAIN, &never) && leader) fail();
      } else if (warp == 1) {
        // -------------------------------------------------------- word of this CTA's operands
        for (uint32_t it = 0; it < total; ++it) {
          if (!mbar_wait(&ctl.full[s], phase, a.wait, abort_flag)) {
            if (leader) fail();
            break;
          }
          if (leader) mbar_arrive_first(first_cta(&ctl.full[s]));
          __syncwarp();
          if (++s == STAGES) s = 0, phase ^= 1;
        }
      }
    }
    if (warp == 2 && lane == 0) {
      // ---------------------------------------------------------- scales (one thread). Not loads of the
      // epilogue's own: its arrival on tempty would wait for those that are on their way (250 cycles a
      // k-block with four of them every fourth)
      pdl_wait();  // the rows' scales
      uint32_t issued = 0, g = 0, phase = 1;
      bool ok = true;
      for (Walk v(tiles, pair, pairs, KB); v.more() && ok; v.advance()) {
        const Tile t = tile_at(ctl.groups, a.E, v.tile, rank);
        const float* xs = a.act_s + (static_cast<size_t>(t.row0 / BM) * KB + v.kb0) * BM;
        const float* ws = a.ws + t.e * a.ws_stride;
        const float *w0, *w1;
        if (GATED) {
          w0 = w1 = ws + static_cast<size_t>(t.n) * scale_stride(KB, 2);
        } else {
          w0 = ws + static_cast<size_t>(2 * t.n) * scale_stride(KB, 1);
          w1 = ws + static_cast<size_t>(min(2 * t.n + 1, NT - 1)) * scale_stride(KB, 1);
        }
        for (int kb = v.kb0; kb < v.kb1; kb += SB) {
          if (!mbar_wait(&ctl.sempty[g], phase, a.wait, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          const int n = min(SB, v.kb1 - kb);
          Scales& sc = ctl.scales[g];
          mbar_arrive_expect_tx(&ctl.sfull[g], n * BM * 4 + 2 * SB * 4);
          bulk_load(sc.x, xs, n * BM * 4, &ctl.sfull[g]);
          xs += SB * BM;
          if (GATED) {
            bulk_load(sc.w, w0 + 2 * kb, 2 * SB * 4, &ctl.sfull[g]);
          } else {
            bulk_load(sc.w, w0 + kb, SB * 4, &ctl.sfull[g]);
            bulk_load(sc.w + SB, w1 + kb, SB * 4, &ctl.sfull[g]);
          }
          ++issued;
          if (++g == SRING) g = 0, phase ^= 1;
        }
      }
      const uint32_t lo = issued > SRING ? issued - SRING : 0;
      for (uint32_t i = lo; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.sfull[i % SRING], (i / SRING) & 1u, Q_DRAIN, &never)) {
          fail();
          break;
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
    // ------------------------------------------------------------ epilogue (warps 4..11)
    pdl_wait();  // what this kernel writes may still be read by the one before
    pdl_trigger();
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * q + lane;  // row of the tile
    // this thread's columns: two runs of 64, of either CTA's part of the matrix tile. Gated: gate and up of
    // channels [64 half, 64 half + 64); else outputs [64 half, 64 half + 64) of tiles 2 n and 2 n + 1
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + 128u * half;
    const uint32_t tempty0 = first_cta(&ctl.tempty[half][0]), tempty1 = first_cta(&ctl.tempty[half][1]);
    uint32_t b = 0, tphase = 0, g = 0, gphase = 0;
    int parity = 0;
    // Once a wait has run out the rest of the tile is gone through without waiting, and nobody is told that a buffer or
    // scales have been read. Where the eight warps meet at a barrier anyway, all leave together; a whole plain tile has
    // none, so there a warp goes on without storing, to where a split tile's barriers count on it.
    bool ok = true;
    for (Walk v(tiles, pair, pairs, KB); v.more(); v.advance(), parity ^= 1) {
      const Tile t = tile_at(ctl.groups, a.E, v.tile, rank);
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb = v.kb0; kb < v.kb1; kb += SB) {
        ok = ok && mbar_wait(&ctl.sfull[g], gphase, a.wait, abort_flag);
        const float* xg = &ctl.scales[g].x[0][r];
        const float* wg = ctl.scales[g].w;
        const int n = min(SB, v.kb1 - kb);
        float f0 = xg[0] * wg[0], f1 = xg[0] * wg[GATED ? 1 : SB];
#pragma unroll 1
        for (int j = 1; j <= n; ++j) {
          // the next k-block's scales are read before this one's product is waited for
          const int jn = j & (SB - 1);
          const float x = xg[jn * BM], w0 = wg[GATED ? 2 * jn : jn], w1 = wg[GATED ? 2 * jn + 1 : SB + jn];
          ok = ok && mbar_wait(&ctl.tfull[half][b], tphase, a.wait, abort_flag);
          tc_fence_after();
          const uint32_t taddr = lane_base + b * 256u;
          // sixteen columns on their way while the sixteen before are added: more in flight would not fit beside
          // the 128 sums
          uint32_t d[2][16];
          tmem_load(taddr, d[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_wait(d[c & 1]);
            if (c < 7) {
              tmem_load(taddr + 16 * (c + 1), d[(c + 1) & 1]);
            } else {
              tc_fence_before();
              __syncwarp();
              if (ok && lane == 0) mbar_arrive_first(b ? tempty1 : tempty0);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              fma2(acc[8 * c + i], __uint_as_float(d[c & 1][2 * i]), __uint_as_float(d[c & 1][2 * i + 1]), c < 4 ? f0 : f1);
          }
          f0 = x * w0, f1 = x * w1;
          b ^= 1u;
          tphase ^= b ^ 1u;
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&ctl.sempty[g]);
        if (++g == SRING) g = 0, gphase ^= 1;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) fail();
      if (v.kb1 - v.kb0 < KB) {
        // a part of the tile, [half][column][row]. Slot 0 of this CTA holds one that starts within its tile, slot 1
        // one that starts it: a run has at most one of each.
        if (epi_any<256>(!ok)) break;  // all eight warps go on, or none
        constexpr size_t slot = 256 * BM;
        const size_t at = static_cast<size_t>(half) * 128 * BM + r;
        float* part = a.parts + (2 * static_cast<size_t>(blockIdx.x) + (v.kb0 == 0 ? 1 : 0)) * slot + at;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          __stcg(part + 2 * i * BM, acc[i].x);
          __stcg(part + (2 * i + 1) * BM, acc[i].y);
        }
        const int first = (v.tile - v.first_split) * v.KG;  // the tile's first unit
        const int c0 = v.holder(first), c1 = v.holder(first + v.KG - 1);
        unsigned* done = a.done + 2 * (v.tile - v.first_split) + rank;
        epi_any<256>(false);
        if (threadIdx.x == 128) {
          __threadfence();  // of what all threads of the barrier have written
          ctl.last = atomicAdd(done, 1u) == static_cast<unsigned>(c1 - c0) ? 1 : 0;
          __threadfence();
        }
        epi_any<256>(false);
        if (!ctl.last) continue;  // (the next write to it comes after another barrier)
        if (threadIdx.x == 128) *done = 0;
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = c0; c <= c1; ++c) {
          const float* p = a.parts + (2 * static_cast<size_t>(2 * c + rank) + (v.start(c) <= first ? 1 : 0)) * slot + at;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            acc[i].x += __ldcg(p + 2 * i * BM);
            acc[i].y += __ldcg(p + (2 * i + 1) * BM);
          }
        }
      } else if (!GATED && !ok) {
        continue;
      }
      const bool valid = r < t.rows;
      const int row = t.row0 + r;
      if (GATED) {
        float am = __uint_as_float(AMAX_MIN_BITS);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          acc[j].x = silu_mul(acc[j].x, acc[32 + j].x);
          acc[j].y = silu_mul(acc[j].y, acc[32 + j].y);
          am = max_abs(am, acc[j].x, acc[j].y);
        }
        // the block of 128 channels is shared with the thread of the other half
        ctl.amax[parity][half][r] = am;
        if (epi_any<256>(!ok)) break;  // all eight warps go on, or none
        am = max_abs(am, ctl.amax[parity][half ^ 1][r], 0.f);
        if (valid) {
          const BlockRatio ratio(am);
          uint8_t* hp = a.h + (static_cast<size_t>(row / BM) * NT + t.n) * A_BYTES;
          // chunks 2 c and 2 c + 1 of a row lie in one 32-byte sector, in the order that the swizzle gives
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 lo = e4m3x16(reinterpret_cast<const float*>(acc) + 32 * c, ratio);
            const uint4 hi = e4m3x16(reinterpret_cast<const float*>(acc) + 32 * c + 16, ratio);
            st_sector(hp + (image_at(r, 64 * half + 32 * c) & ~31u), (r & 1) ? hi : lo, (r & 1) ? lo : hi);
          }
          if (half == 0) a.h_s[(static_cast<size_t>(row / BM) * NT + t.n) * BM + r] = block_scale(am);
        }
      } else {
        // Through shared memory, 128 bytes of each of the warp's 32 rows at a time: then eight lanes have a row's, and a
        // store is four whole lines. As 32 bytes of every lane's own row it was 32 pieces of lines (256 fp32 columns,
        // 3.1 us a tile).
        uint4(*buf)[8] = reinterpret_cast<uint4(*)[8]>(smem + STAGES * STAGE + (warp - 4) * (32 * 128));
        const int size = a.out_f32 ? 4 : 2, n16 = a.out_f32 ? 2 : 1;  // bytes of a value, 128-byte pieces of 64 columns
        const bool even = a.ldy * size % 16 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const int col = 256 * t.n + 128 * part + 64 * half;
          const int cols = min(64, a.N - col);
          if (cols <= 0) break;
          const float2* v = acc + 32 * part;
          if (even && cols == 64) {
            uint8_t* y = static_cast<uint8_t*>(a.y) + (static_cast<size_t>(t.row0 + 32 * q) * a.ldy + col) * size;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c >= n16) break;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint4 w;
                if (a.out_f32) {
                  const float2 p0 = v[16 * c + 2 * i], p1 = v[16 * c + 2 * i + 1];
                  w = make_uint4(__float_as_uint(p0.x), __float_as_uint(p0.y), __float_as_uint(p1.x), __float_as_uint(p1.y));
                } else {
                  const float2* p = v + 4 * i;
                  w = make_uint4(pack_bf16x2(p[0].x, p[0].y), pack_bf16x2(p[1].x, p[1].y), pack_bf16x2(p[2].x, p[2].y),
                                 pack_bf16x2(p[3].x, p[3].y));
                }
                buf[lane][i ^ (lane & 7)] = w;
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int row = 4 * i + (lane >> 3), piece = lane & 7;
                if (32 * q + row < t.rows)
                  *reinterpret_cast<uint4*>(y + static_cast<size_t>(row) * a.ldy * size + 128 * c + 16 * piece) =
                      buf[row][piece ^ (row & 7)];
              }
              __syncwarp();
            }
          } else if (valid) {
            const size_t o = static_cast<size_t>(row) * a.ldy + col;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (a.out_f32) {
                float* y = static_cast<float*>(a.y) + o;
                if (2 * j < cols) y[2 * j] = v[j].x;
                if (2 * j + 1 < cols) y[2 * j + 1] = v[j].y;
              } else {
                uint16_t* y = static_cast<uint16_t*>(a.y) + o;
                const uint32_t w = pack_bf16x2(v[j].x, v[j].y);
                if (2 * j < cols) y[2 * j] = static_cast<uint16_t>(w);
                if (2 * j + 1 < cols) y[2 * j + 1] = static_cast<uint16_t>(w >> 16);
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  cluster_sync();  // nothing of either CTA is still used by the other
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace

size_t qgemm_wide_parts(int num_sms) { return static_cast<size_t>(2) * num_sms * 256 * BM; }

cudaError_t launch_qgemm_wide(const QGemmArgs& a, bool gated, cudaStream_t st) {
  const size_t smem = STAGES * STAGE + (gated ? 0 : OUT_BYTES) + 1024;
  const void* k = gated ? reinterpret_cast<const void*>(&k_qgemm_wide<true>) : reinterpret_cast<const void*>(&k_qgemm_wide<false>);
  const cudaError_t e = ensure_dyn_smem(k, smem);
  if (e != cudaSuccess) return e;
  return gated ? launch_q(k_qgemm_wide<true>, dim3(a.num_sms & ~1), THREADS, smem, st, a)
               : launch_q(k_qgemm_wide<false>, dim3(a.num_sms & ~1), THREADS, smem, st, a);
}

}  // namespace pop
