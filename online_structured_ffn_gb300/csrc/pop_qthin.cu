// Products of few rows (tokens) and a matrix in e4m3 with block scales: the matrix streams once.
//
// y[n][f] = sum over k-blocks b of s_x[n][b] s_w[f/128][b] * (q_x[n] . q_w[f])_b. The matrix is the M operand
// (128 outputs f per tile), the tokens the N operand (NT = 16, 32 or 64 per tile, as many as there are,
// rounded up to 16). A k-block is one tcgen05 product of 128 x N x 128 into TMEM columns of its own,
// which the epilogue adds to fp32 registers with the block's scales; a stage's two products (two k-blocks, or the
// gate's and the up's of one) make one TMEM buffer. Bound by the matrix's bytes, so the
// split is one that keeps every SM streaming to the end: all (tile, k-block) pairs in order are cut into
// one equal run per CTA. A tile that lies in several runs is summed from fp32 parts in the order of k by
// whichever of its CTAs comes last (a counter per tile; no CTA waits for another), so the bits do not
// depend on the order in which CTAs run.
//
// Up to 16 rows of one group need no kernel before this one: with ROWS, warps 10..17 bring each stage's rows from
// bf16 (or e4m3) into their image themselves. Every CTA does so for the k-blocks of its run, which is little beside
// the matrix's bytes (16 rows: 4 KB of 20 a k-block, from L2), and saves the quantiser's launch (one row by 11008 x
// 4096: 17 us a call with it, 12.3 without).
//
// Warp 0: copies. A stage is 32 KB of the matrix (one bulk copy: its image is what shared memory needs) and the same
// k-blocks of the rows and of their scales (a copy each; a run of rows is one tile). The matrix does not depend on
// the kernel before, so the first stages' copies of it go out before this one is waited for. Warp 1: products. Warps
// 2..9: epilogue, TMEM lane quarter warp % 4, two warps to a quarter that have its rows in turn. Every wait has a limit;
// a CTA that gives up records QERR_TIMEOUT, lets its copies and products finish, frees TMEM and returns.
//
// A tile in several runs costs its CTA 6 to 10 thousand cycles: the part on its way out, a fence and the counter 2500,
// the sum 2000 to 5000. So the part of a run's first tile is handed in by a warp of its own, the last, while the
// epilogue goes on (11008 x 4096 with one row 12.0 -> 11.0 us), and that warp then looks out for the others' parts of the
// run's last tile: where they are all there in time, as they mostly are, the epilogue adds them to its registers
// and hands nothing in (64 x (2 x 1000 x 2048) with 31 rows each 50.4 -> 46.9 us).
//
// Measured, back to back: 8 x (2 x 14336 x 4096) with 8 rows each 132 us (7.1 TB/s of the matrices' bytes), 8 x 4096 x
// 14336 68.7 (6.8), 8192 x 28672 with 16 rows 39 (6.0), 2 x (2 x 14336 x 4096) with one row 36.6 (6.4), 11008 x 4096 with
// one row 10.8 (4.2); 64 x (2 x 1000 x 2048) with 31 rows 46.9 (5.7) and 64 x 2048 x 1000 28.8 (4.7), where a tile's end
// comes every 16 or 8 k-blocks and takes some 2000 cycles of the epilogue.
#include "pop_qdevice.cuh"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int THREADS = 320, EPI = 256, HAND = 32;
constexpr uint32_t RING_BYTES = 220 * 1024;
constexpr uint32_t TMEM_COLS = 512;
// More in flight is slower, not faster (8 x 2 x 14336 x 4096: 132 us with 4 stages, 135 with 5, 134 with 3; 64 x 2 x 1000 x
// 2048 with 64 rows 50.3, 50.3 and 49.7).
constexpr int MAX_STAGES = 4, MAX_BUFS = 8;

template <bool GATED, int NT>
struct Thin {
  static constexpr int P = GATED ? 2 : 1;
  static constexpr int KS = GATED ? 1 : 2;          // k-blocks of a stage
  static constexpr uint32_t W_BYTES = P * QTILE;    // of a k-block
  static constexpr uint32_t X_BYTES = NT * QB;      // of a k-block's rows: one run of NT
  static constexpr uint32_t S_BYTES = NT * 4;       // of their scales
  static constexpr uint32_t X_OFF = KS * W_BYTES;
  static constexpr uint32_t STAGE = X_OFF + KS * X_BYTES;
  static constexpr uint32_t H_BYTES = NT * QB * 4;  // a finished tile on its way out
  static constexpr int FIT = (RING_BYTES - H_BYTES) / STAGE;
  static constexpr int STAGES = FIT < MAX_STAGES ? FIT : MAX_STAGES;
  static constexpr int BUFS = static_cast<int>(TMEM_COLS) / (2 * NT) < MAX_BUFS ? static_cast<int>(TMEM_COLS) / (2 * NT) : MAX_BUFS;
  // The rows' scales have a ring of their own, as the epilogue needs them for longer than the products need a stage.
  // A stage's products wait for the buffer BUFS before, and its copies for the products STAGES before, so what a slot
  // held SLOTS stages ago has been read.
  static constexpr int SLOTS = STAGES + BUFS;
  static constexpr uint32_t SLOT = KS * S_BYTES;
  static constexpr uint32_t S_OFF = STAGES * STAGE + H_BYTES;  // of the slots, behind the ring and the tile
  static constexpr uint32_t SMEM = S_OFF + SLOTS * SLOT + 1024;
  static_assert(STAGE % 1024 == 0 && STAGES <= MAX_STAGES, "images start on 1 KB");
};

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t sfull[MAX_STAGES + MAX_BUFS];
  uint64_t tfull[MAX_BUFS], tempty[MAX_BUFS];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int last;
  int late, late_tile, late_t, late_rows, late_run;  // a first part: whether it was its tile's last, and the tile
  int others, alone;  // the last tile: whether the others' parts are there; as the epilogue saw it
  int over;           // the epilogue needs no news of it any more
  Groups groups;
};

// The tiles of one CTA's run of (tile, k-block) units [x0, x1), in order, each with its k-blocks.
template <int NT>
struct Walk {
  int tile, kb0, kb1;
  int e, t, n;  // group, output tile, rows of the tile
  int run;      // of rows
  __device__ __forceinline__ Walk(const Groups& gr, int E, int KB, long long x0, long long x1) : gr_(gr), KB_(KB) {
    tile = static_cast<int>(x0 / KB);
    kb0 = static_cast<int>(x0 - static_cast<long long>(tile) * KB);
    left_ = static_cast<int>(x1 - x0);
    if (left_ <= 0) return;
    e = gr.of(E, tile);
    enter();
    const int local = tile - gr.tile0[e];
    t = local / tts_;  // the row tiles of one output tile side by side: the matrix tile is in L2 for the others
    i_ = local - t * tts_;
    place();
  }
  __device__ __forceinline__ bool more() const { return left_ > 0; }
  __device__ __forceinline__ void next() {
    left_ -= kb1 - kb0;
    if (left_ <= 0) return;
    kb0 = 0;
    ++tile;
    if (++i_ == tts_) i_ = 0, ++t;
    if (tile == gr_.tile0[e + 1]) {
      do ++e;
      while (tile == gr_.tile0[e + 1]);  // groups without rows
      enter();
      t = i_ = 0;
    }
    place();
  }

 private:
  const Groups& gr_;
  int KB_, left_, tts_, i_, cnt_, run0_;
  __device__ __forceinline__ void enter() {
    cnt_ = gr_.count[e];
    run0_ = gr_.run0[e];
    tts_ = qceil(cnt_, NT);
  }
  __device__ __forceinline__ void place() {
    kb1 = min(KB_, kb0 + left_);
    n = min(NT, cnt_ - i_ * NT);
    run = run0_ + i_;
  }
};

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(EPI) : "memory"); }

// Barriers 2 (the first part is written) and 3 (it is handed in) of the epilogue's warps and the one that hands it in.
template <int B>
__device__ __forceinline__ void hand_sync() { asm volatile("bar.sync %0, %1;" ::"n"(B), "n"(EPI + 32) : "memory"); }
template <int B>
__device__ __forceinline__ void hand_arrive() { asm volatile("bar.arrive %0, %1;" ::"n"(B), "n"(EPI + 32) : "memory"); }

// The quotient of two numbers that are not negative, b > 0: by 32 bits where those hold them.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

constexpr int LOOKS = 1 << 17;  // for others' parts, 0.3 us or more apart
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One more part of a tile is there, written by threads that have met at a barrier. Whether it was the last of `parts`.
__device__ __forceinline__ bool hand_in(unsigned* done, int parts) {
  __threadfence();
  const bool last = atomicAdd(done, 1u) == static_cast<unsigned>(parts - 1);
  __threadfence();
  if (last) *done = 0;
  return last;
}

constexpr int ROW_TEAM = 128, ROW_TEAMS = 2, ROW_THREADS = ROW_TEAM * ROW_TEAMS;  // beside the others, with ROWS

template <bool GATED, int NT, bool ROWS>
__global__ void __launch_bounds__(THREADS + (ROWS ? ROW_THREADS : 0) + HAND, 1)
    k_qgemm_thin(const __grid_constant__ QGemmArgs a, const __grid_constant__ QRowsArgs in) {
  using C = Thin<GATED, NT>;
  constexpr int P = C::P, HAND_WARP = (THREADS + (ROWS ? ROW_THREADS : 0)) / 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int KB = qceil(a.K, QB), NTILES = qceil(a.N, QB);
  volatile int* abort_flag = &ctl.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&ctl.full[s], 1 + (ROWS ? ROW_TEAM / 32 : 0));
      mbar_init(&ctl.empty[s], 1);
    }
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&ctl.sfull[i], ROWS ? ROW_TEAM / 32 : 1);
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(&ctl.tfull[b], 1);
      mbar_init(&ctl.tempty[b], EPI / 32);
    }
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = ctl.others = ctl.over = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  ctl.groups.zero(a);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base;
  // The groups' numbers, or the experts that they are counted from, are two kernels back or more: the kernel before this
  // waited for them before it let this one start (as this one does: pdl_trigger comes after a pdl_wait).
  const int tiles = ctl.groups.fill<true>(a, NT, NTILES);
  const long long work = static_cast<long long>(tiles) * KB;
  // CTAs that have a run, G: all, but with few tiles a run is at least sqrt(NT KB / 28) units, as each more CTA of a
  // tile costs its last one the reading of a part (NT = 64: some 0.8 us; a unit takes 0.35 us). Runs that are whole
  // fractions of a tile have one part to hand in instead of two, which is worth some six units. (64 rows by 1000 x
  // 8000: 29 us over all 152 CTAs, 19 to a tile, 18 by the square root alone.)
  const int least = max(1, static_cast<int>(sqrtf(NT * KB / 28.f)));
  const int spread = static_cast<int>(min(static_cast<long long>(gridDim.x), max(work / least, min(work, 1ll))));
  const int each = tiles > 0 ? min(static_cast<int>(gridDim.x) / tiles, max(1, KB / least)) : 0;  // CTAs to a tile
  const bool aligned = each > 0 && qceil(KB, each) <= work / spread + 6;
  const long long G = aligned ? static_cast<long long>(tiles) * each : spread;
  const bool on = static_cast<long long>(blockIdx.x) < G;
  const long long x0 = on ? work * blockIdx.x / G : 0, x1 = on ? work * (blockIdx.x + 1) / G : 0;

  // The first tile of this run is in others too, and there are more tiles: its part is handed in by a warp of its own.
  const auto hand = [&]() {
    const long long tile = quotient(x0, KB);
    return x0 < x1 && tile * KB != x0 && (tile + 1) * KB < x1;
  };
  // The CTAs that share a tile. CTA c holds [work c / G, work (c + 1) / G): the one of unit x is ((x + 1) G - 1) / work.
  const auto first_cta_of = [&](int tile) { return static_cast<int>(quotient((static_cast<long long>(tile) * KB + 1) * G - 1, work)); };
  const auto last_cta_of = [&](int tile) { return static_cast<int>(quotient((static_cast<long long>(tile) + 1) * KB * G - 1, work)); };

  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      atomicOr(a.err, QERR_TIMEOUT);
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- copies (one thread)
      // A stage's rows follow its part of the matrix; the first stages' all at once, after the wait.
      struct Rows {
        const uint8_t* x;
        const float* s;
        int n;  // k-blocks
      } owed[C::STAGES];
      auto load_rows = [&](const Rows& r, uint32_t s, uint32_t slot) {
        bulk_load(smem + s * C::STAGE + C::X_OFF, r.x, r.n * C::X_BYTES, &ctl.full[s]);
        mbar_arrive_expect_tx(&ctl.sfull[slot], r.n * C::S_BYTES);
        bulk_load(smem + C::S_OFF + slot * C::SLOT, r.s, r.n * C::S_BYTES, &ctl.sfull[slot]);
      };
      uint32_t issued = 0, s = 0, phase = 1, slot = 0;
      bool ok = true, waited = ROWS;
      for (Walk<NT> g(ctl.groups, a.E, KB, x0, x1); g.more() && ok; g.next()) {
        const uint8_t* w = a.w + g.e * a.w_stride + (static_cast<size_t>(g.t) * KB + g.kb0) * C::W_BYTES;
        Rows r;
        r.x = a.act + (static_cast<size_t>(g.run) * KB + g.kb0) * C::X_BYTES;
        r.s = a.act_s + (static_cast<size_t>(g.run) * KB + g.kb0) * NT;
        for (int kb = g.kb0; kb < g.kb1; kb += C::KS) {
          if (!waited && issued == C::STAGES) {
            pdl_wait();
            waited = true;
#pragma unroll
            for (int i = 0; i < C::STAGES; ++i) load_rows(owed[i], i, i);
          }
          if (!mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          r.n = min(C::KS, g.kb1 - kb);
          mbar_arrive_expect_tx(&ctl.full[s], r.n * (C::W_BYTES + (ROWS ? 0 : C::X_BYTES)));
          bulk_load(smem + s * C::STAGE, w, r.n * C::W_BYTES, &ctl.full[s]);
          if (waited) {
            if (!ROWS) load_rows(r, s, slot);
          } else {
#pragma unroll
            for (int i = 0; i < C::STAGES; ++i)
              if (i == static_cast<int>(s)) owed[i] = r;
          }
          w += C::KS * C::W_BYTES;
          r.x += C::KS * C::X_BYTES;
          r.s += C::KS * NT;
          ++issued;
          if (++s == C::STAGES) s = 0, phase ^= 1;
          if (++slot == C::SLOTS) slot = 0;
        }
      }
      if (!waited) {  // a short run: every stage that was begun gets its rows
        pdl_wait();
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i)
          if (i < static_cast<int>(issued)) load_rows(owed[i], i, i);
      }
      // no copy of this CTA may be in flight when it exits
      const uint32_t lo = issued > C::STAGES ? issued - C::STAGES : 0;
      for (uint32_t i = lo; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.full[i % C::STAGES], (i / C::STAGES) & 1u, Q_DRAIN, &never)) {
          fail();
          break;  // (with ROWS it waits for rows that nobody brings; the copies have had their time)
        }
      }
      for (uint32_t i = ROWS ? issued : issued > C::SLOTS ? issued - C::SLOTS : 0; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.sfull[i % C::SLOTS], (i / C::SLOTS) & 1u, Q_DRAIN, &never)) {
          fail();
          break;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products (one warp, one lane of it issuing)
    const bool leader = elect_one();
    const uint32_t ring = desc_lo(smem_u32(smem));
    uint32_t s = 0, phase = 0, b = 0, tphase = 1;
    bool ok = true;
    for (Walk<NT> g(ctl.groups, a.E, KB, x0, x1); g.more() && ok; g.next()) {
      const uint32_t idesc = idesc_e4m3_f32(128, qceil(g.n, 16) * 16);
      for (int kb = g.kb0; kb < g.kb1 && ok; kb += C::KS) {
        ok = mbar_wait(&ctl.full[s], phase, a.wait, abort_flag) && mbar_wait(&ctl.tempty[b], tphase, a.wait, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t st = ring + s * (C::STAGE >> 4);
          const uint32_t d = tmem_base + b * static_cast<uint32_t>(2 * NT);
          umma_block(d, st, st + (C::X_OFF >> 4), idesc);
          if (GATED)
            umma_block(d + NT, st + (QTILE >> 4), st + (C::X_OFF >> 4), idesc);
          else if (kb + 1 < g.kb1)
            umma_block(d + NT, st + (QTILE >> 4), st + ((C::X_OFF + C::X_BYTES) >> 4), idesc);
          umma_commit(&ctl.tfull[b]);
          umma_commit(&ctl.empty[s]);
        }
        __syncwarp();
        if (++b == C::BUFS) b = 0, tphase ^= 1;
        if (++s == C::STAGES) s = 0, phase ^= 1;
      }
    }
    if (!ok && leader) fail();
    if (leader) umma_commit(&ctl.drain);
    volatile int never = 0;
    if (!mbar_wait(&ctl.drain, 0, Q_DRAIN, &never) && leader) fail();
    __syncwarp();
  } else if (ROWS && warp >= 10 && warp < HAND_WARP) {
    // ------------------------------------------------------------ rows (warps 10..17): eight lanes to a row, two teams
    // in turn: a stage takes a team about 1900 cycles from its loads to its arrival, and the matrix comes in 1400
    pdl_wait();
    const int team = (threadIdx.x - THREADS) / ROW_TEAM;
    const int row = ((threadIdx.x - THREADS) & (ROW_TEAM - 1)) >> 3, lane8 = threadIdx.x & 7;
    const bool mine = row < in.M;
    // A stage's values: of its two k-blocks, 16 of bf16 each, or of e4m3 in the first half.
    struct Raw {
      uint4 v[2][2];
      float scale[2];
    };
    auto load = [&](Raw& raw, int kb, int n) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k0 = (kb + u) * QB + lane8 * 16;
        const int n8 = mine && u < n ? min(max((in.K - k0) >> 3, 0), 2) : 0;
        raw.v[u][0] = raw.v[u][1] = make_uint4(0u, 0u, 0u, 0u);
        raw.scale[u] = 0.f;
        if (in.kind == 0) {
          const uint16_t* p = static_cast<const uint16_t*>(in.x) + static_cast<size_t>(row) * in.ldx + k0;
          if (n8 > 0) raw.v[u][0] = __ldg(reinterpret_cast<const uint4*>(p));
          if (n8 > 1) raw.v[u][1] = __ldg(reinterpret_cast<const uint4*>(p + 8));
        } else {
          const uint8_t* p = static_cast<const uint8_t*>(in.x) + static_cast<size_t>(row) * in.ldx + k0;
          if (n8 > 0) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            raw.v[u][0].x = v.x, raw.v[u][0].y = v.y;
          }
          if (n8 > 1) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p + 8));
            raw.v[u][0].z = v.x, raw.v[u][0].w = v.y;
          }
          if (mine && u < n) raw.scale[u] = __ldg(in.xs + static_cast<size_t>(row) * in.lds + kb + u);
        }
      }
    };
    auto write = [&](const Raw& raw, uint8_t* st, uint8_t* scales) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 q = raw.v[u][0];
        float sc = raw.scale[u];
        if (in.kind == 0) {
          const uint4 a0 = raw.v[u][0], a1 = raw.v[u][1];
          const uint32_t w[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
          float v[16];
          float am = __uint_as_float(AMAX_MIN_BITS);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] = bf16lo(w[i]), v[2 * i + 1] = bf16hi(w[i]);
            am = max_abs(am, v[2 * i], v[2 * i + 1]);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) am = max_abs(am, __shfl_xor_sync(0xffffffffu, am, o), 0.f);
          q = e4m3x16(v, BlockRatio(am));
          sc = block_scale(am);
        }
        if (mine) {
          *reinterpret_cast<uint4*>(st + C::X_OFF + u * C::X_BYTES + image_at(row, lane8 * 16)) = q;
          if (lane8 == 0) *reinterpret_cast<float*>(scales + u * C::S_BYTES + row * 4) = sc;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the products read what was written here
    };
    Raw raw;
    Walk<NT> g(ctl.groups, a.E, KB, x0, x1);
    int kb = g.kb0;
    auto step = [&]() {  // to the next stage
      kb += C::KS;
      if (kb >= g.kb1) {
        g.next();
        kb = g.kb0;
      }
    };
    uint32_t s = 0, phase = 1, slot = 0;
    auto ring_step = [&]() {
      if (++s == C::STAGES) s = 0, phase ^= 1;
      if (++slot == C::SLOTS) slot = 0;
    };
    bool ok = true;
    for (int i = 0; i < team && g.more(); ++i) step(), ring_step();
    if (g.more()) load(raw, kb, g.kb1 - kb);
    while (g.more()) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag));
      if (!ok) break;
      write(raw, smem + s * C::STAGE, smem + C::S_OFF + slot * C::SLOT);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.full[s]);
        mbar_arrive(&ctl.sfull[slot]);
      }
#pragma unroll
      for (int i = 0; i < ROW_TEAMS; ++i) {
        ring_step();
        if (g.more()) step();
      }
      if (g.more()) load(raw, kb, g.kb1 - kb);
    }
    if (!ok && lane == 0) fail();
  } else if (warp == HAND_WARP) {
    // ------------------------------------------------------------ a first part is handed in
    if (hand()) {
      const int tile = static_cast<int>(quotient(x0, KB));
      const int parts = last_cta_of(tile) - first_cta_of(tile) + 1;
      pdl_wait();
      hand_sync<2>();
      if (lane == 0) ctl.late = !*abort_flag && hand_in(a.done + tile, parts) ? 1 : 0;
      __syncwarp();
      hand_arrive<3>();
    }
    // The last tile, if this CTA has its beginning and others the rest: looks out for their parts, so that the
    // epilogue, where all are there when it is done, adds them to its own registers and hands nothing in.
    const long long end = quotient(x1, KB);
    if (x0 <= end * KB && end * KB < x1) {
      const int tile = static_cast<int>(end), others = last_cta_of(tile) - static_cast<int>(blockIdx.x);
      pdl_wait();
      if (lane == 0) {
        for (int i = 0; i < LOOKS && !*static_cast<volatile int*>(&ctl.over); ++i) {
          if (ld_acquire(a.done + tile) == static_cast<unsigned>(others)) {
            __threadfence_block();
            *static_cast<volatile int*>(&ctl.others) = 1;
            break;
          }
          __nanosleep(300);
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9)
    pdl_wait();  // what this kernel writes may still be read by the one before
    pdl_trigger();
    // The tile's rows are in chunks of CH that the two warps of a quarter have in turn (so that both have some where
    // a tile is half empty); chunk c of a thread begins at row n0 + 2 CH c.
    constexpr int CW = NT / 2, CH = NT == 64 ? 16 : 8, NC = CW / CH;
    const int q = warp & 3, n0 = CH * ((warp - 2) >> 2);
    const int f = 32 * q + lane;  // output of the tile
    const int et = threadIdx.x - 64;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + n0;
    uint32_t slot = 0, sphase = 0, b = 0, tphase = 0;
    // The matrix's scales of a run of k-blocks: lane i holds number 32 j + i, and the one after is on its way; the
    // next tile's first while this one is written out.
    Walk<NT> g(ctl.groups, a.E, KB, x0, x1);
    const float* ws = nullptr;
    int nw = 0;
    float sw_next = 0.f;
    auto first_scales = [&]() {
      ws = a.ws + g.e * a.ws_stride + static_cast<size_t>(g.t) * scale_stride(KB, P) + g.kb0 * P;
      nw = (g.kb1 - g.kb0) * P;
      sw_next = lane < nw ? __ldg(ws + lane) : 0.f;
    };
    if (g.more()) first_scales();
    bool owed = hand(), handed = false;  // the first part: still to be written; handed in, and not seen after yet
    // A finished tile goes through shared memory, hs[row][output], so that it leaves in whole 16-byte pieces by
    // short loops: as unrolled stores of every thread's own column it took several thousand cycles a tile.
    float* hs = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
    // A part of a tile is [product][row][output]. Slot 0 of a CTA holds one that starts within its tile, slot 1
    // one that starts it: a run has at most one of each.
    constexpr size_t PART = static_cast<size_t>(P) * NT * QB;
    // The CTAs that share a tile, and whether the first one's part starts it (the others' lie within).
    int c0 = 0, c1 = 0;
    bool whole0 = false;
    auto sharers = [&](int tile) {
      c0 = first_cta_of(tile), c1 = last_cta_of(tile);
      whole0 = quotient(work * c0, G) <= static_cast<long long>(tile) * KB;
    };
    while (true) {
      int tile, t, rows;
      size_t run;
      bool join;
      if (g.more()) {
        float sw = 0.f;
        const int nc = min(NC, qceil(max(g.n - n0, 0), 2 * CH));  // chunks with rows
        float2 acc[P][NC][CH / 2];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < CH / 2; ++j) acc[p][c][j] = make_float2(0.f, 0.f);
        // once a wait has run out the rest of the run is gone through without waiting, and nobody is told that a
        // buffer has been read
        bool ok = true;
        int i = 0;
        for (int kb = g.kb0; kb < g.kb1; kb += C::KS) {
          if ((i & 31) == 0) {
            sw = sw_next;
            sw_next = i + 32 + lane < nw ? __ldg(ws + i + 32 + lane) : 0.f;
          }
          // the two products' scales; a k-block that is not there (the last of an odd number) gets 0 times what its
          // columns hold, which is left out below
          const float s0 = __shfl_sync(0xffffffffu, sw, i & 31), s1 = __shfl_sync(0xffffffffu, sw, (i + 1) & 31);
          i += 2;
          const bool two = GATED || kb + 1 < g.kb1;
          const float4* sx0 = reinterpret_cast<const float4*>(smem + C::S_OFF + slot * C::SLOT + n0 * 4);
          const float4* sx1 = sx0 + (GATED ? 0 : C::S_BYTES / 16);
          const uint32_t taddr = lane_base + b * static_cast<uint32_t>(2 * NT);
          ok = ok && mbar_wait(&ctl.sfull[slot], sphase, a.wait, abort_flag) &&
               mbar_wait(&ctl.tfull[b], tphase, a.wait, abort_flag);
          tc_fence_after();
          // (all chunks on their way together where the registers hold them)
          constexpr int LC = GATED && NT == 64 ? 1 : NC;
#pragma unroll
          for (int l0 = 0; l0 < NC; l0 += LC) {
            uint32_t d0[LC][CH], d1[LC][CH];
#pragma unroll
            for (int l = 0; l < LC; ++l) {
              if (l0 + l >= nc) break;
              tmem_load(taddr + 2 * CH * (l0 + l), d0[l]);
              if (two) tmem_load(taddr + NT + 2 * CH * (l0 + l), d1[l]);
            }
#pragma unroll
            for (int l = 0; l < LC; ++l) tmem_wait(d0[l]), tmem_wait(d1[l]);
#pragma unroll
            for (int l = 0; l < LC; ++l) {
              const int c = l0 + l;
              if (c >= nc) break;
#pragma unroll
              for (int j = 0; j < CH / 2; j += 2) {
                const float4 v = sx0[(2 * CH * c + 2 * j) >> 2];
                fma2(acc[0][c][j], d0[l][2 * j], d0[l][2 * j + 1], mul2(s0, v.x, v.y));
                fma2(acc[0][c][j + 1], d0[l][2 * j + 2], d0[l][2 * j + 3], mul2(s0, v.z, v.w));
                if (GATED) {
                  fma2(acc[P - 1][c][j], d1[l][2 * j], d1[l][2 * j + 1], mul2(s1, v.x, v.y));
                  fma2(acc[P - 1][c][j + 1], d1[l][2 * j + 2], d1[l][2 * j + 3], mul2(s1, v.z, v.w));
                }
              }
              if (!GATED && two) {
#pragma unroll
                for (int j = 0; j < CH / 2; j += 2) {
                  const float4 v = sx1[(2 * CH * c + 2 * j) >> 2];
                  fma2(acc[0][c][j], d1[l][2 * j], d1[l][2 * j + 1], mul2(s1, v.x, v.y));
                  fma2(acc[0][c][j + 1], d1[l][2 * j + 2], d1[l][2 * j + 3], mul2(s1, v.z, v.w));
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&ctl.tempty[b]);  // (and the slot of the scales has been read)
          if (++b == C::BUFS) b = 0, tphase ^= 1;
          if (++slot == C::SLOTS) slot = 0, sphase ^= 1;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) fail();
        const bool begins = g.kb0 == 0 && g.kb1 < KB;
        if (begins && et == 0) {
          ctl.alone = *static_cast<volatile int*>(&ctl.others);
          *static_cast<volatile int*>(&ctl.over) = 1;
          __threadfence_block();
        }
        if (epi_any<EPI>(!ok)) break;  // all warps go on, or none
        tile = g.tile, t = g.t, rows = g.n, run = g.run;
        const int kb0 = g.kb0;
        join = g.kb1 - g.kb0 < KB;
        g.next();
        if (g.more()) first_scales();
        if (begins && ctl.alone) {
          // this CTA's part comes first; the others' are added in the order of k, as below (and to 0 first, as there)
          if (et == 0) a.done[tile] = 0;
          join = false;
          const int end = last_cta_of(tile);
          for (int c = blockIdx.x + 1; c <= end; ++c) {
            const float* part = a.parts + 2 * static_cast<size_t>(c) * PART + n0 * QB + f;
#pragma unroll
            for (int l = 0; l < NC; ++l) {
              if (l >= nc) break;
#pragma unroll
              for (int p = 0; p < P; ++p) {
                float w[CH];
#pragma unroll
                for (int j = 0; j < CH; ++j)
                  w[j] = n0 + 2 * CH * l + j < rows ? __ldcg(part + (p * NT + 2 * CH * l + j) * QB) : 0.f;
#pragma unroll
                for (int j = 0; j < CH; j += 2) {
                  float2& v = acc[p][l][j / 2];
                  v = make_float2((v.x + 0.f) + w[j], (v.y + 0.f) + w[j + 1]);
                }
              }
            }
          }
        }
        if (!join) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (c >= nc) break;
#pragma unroll
            for (int j = 0; j < CH / 2; ++j) {
              const float2 v = acc[0][c][j], u = acc[P - 1][c][j];
              float* h = hs + (n0 + 2 * CH * c + 2 * j) * QB + f;
              h[0] = GATED ? silu_mul(v.x, u.x) : v.x;
              h[QB] = GATED ? silu_mul(v.y, u.y) : v.y;
            }
          }
          epi_sync();
        } else {
          float* part = a.parts + (2 * static_cast<size_t>(blockIdx.x) + (kb0 == 0 ? 1 : 0)) * PART + n0 * QB + f;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (c >= nc) break;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
              for (int j = 0; j < CH / 2; ++j) {
                float* at = part + (p * NT + 2 * CH * c + 2 * j) * QB;
                const int left = rows - (n0 + 2 * CH * c + 2 * j);  // (what waits below waits for every store)
                if (left > 0) __stcg(at, acc[p][c][j].x);
                if (left > 1) __stcg(at + QB, acc[p][c][j].y);
              }
          }
          if (owed) {
            // Nobody waits for its tile here: the CTA before this one will mostly be the last one there. If this one was,
            // it has seen to the tile after its others.
            if (et == 0) ctl.late_tile = tile, ctl.late_t = t, ctl.late_rows = rows, ctl.late_run = static_cast<int>(run);
            hand_arrive<2>();
            owed = false, handed = true;
            continue;
          }
          sharers(tile);  // (while the part is on its way out)
          epi_sync();
          if (et == 0) ctl.last = hand_in(a.done + tile, c1 - c0 + 1) ? 1 : 0;
          epi_sync();
          if (!ctl.last) continue;  // (the next write to it comes after another barrier)
        }
      } else if (handed) {
        handed = false;
        hand_sync<3>();
        if (!ctl.late) break;
        tile = ctl.late_tile, t = ctl.late_t, rows = ctl.late_rows, run = ctl.late_run;
        sharers(tile);
        join = true;
      } else {
        break;
      }
      if (join) {
        // all of a part's loads on their way together, as far as the registers hold them: one after the other they
        // took some 1500 cycles each (31 rows, gated: 7000 a tile)
        constexpr int U = NT == 16 ? 1 : GATED ? 2 : 4;
        for (int i0 = et; i0 < rows * (QB / 4); i0 += U * EPI) {
          float4 v[U][P];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int p = 0; p < P; ++p) v[u][p] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
          for (int c = c0; c <= c1; ++c) {
            const float4* p0 =
                reinterpret_cast<const float4*>(a.parts + (2 * static_cast<size_t>(c) + (c == c0 && whole0 ? 1 : 0)) * PART);
            float4 w[U][P];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int p = 0; p < P; ++p)
                if (i0 + u * EPI < rows * (QB / 4)) w[u][p] = __ldcg(p0 + p * NT * (QB / 4) + i0 + u * EPI);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int p = 0; p < P; ++p)
                if (i0 + u * EPI < rows * (QB / 4))
                  v[u][p].x += w[u][p].x, v[u][p].y += w[u][p].y, v[u][p].z += w[u][p].z, v[u][p].w += w[u][p].w;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (i0 + u * EPI >= rows * (QB / 4)) break;
            if (GATED) {
              const float4 g = v[u][0], h = v[u][P - 1];
              v[u][0] = make_float4(silu_mul(g.x, h.x), silu_mul(g.y, h.y), silu_mul(g.z, h.z), silu_mul(g.w, h.w));
            }
            reinterpret_cast<float4*>(hs)[i0 + u * EPI] = v[u][0];
          }
        }
        epi_sync();
      }
      if (!GATED) {
        const size_t o = run * NT * a.ldy + t * QB;
        const size_t size = a.out_f32 ? 4 : 2;
        const bool whole = t * QB + QB <= a.N && a.ldy % 4 == 0 && (o * size + reinterpret_cast<uintptr_t>(a.y)) % (4 * size) == 0;
#pragma unroll 2
        for (int i = et; i < rows * (QB / 4); i += EPI) {
          const int n = i >> 5, c = (i & 31) * 4;
          const float4 v = reinterpret_cast<const float4*>(hs)[i];
          const size_t at = o + static_cast<size_t>(n) * a.ldy + c;
          if (whole && a.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = v;
          } else if (whole) {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          } else {
            const float vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (t * QB + c + j >= a.N) break;
              if (a.out_f32)
                static_cast<float*>(a.y)[at + j] = vs[j];
              else
                static_cast<__nv_bfloat16*>(a.y)[at + j] = __float2bfloat16_rn(vs[j]);
            }
          }
        }
      } else {
        // the tile's 128 channels are one block of the next product's rows: eight lanes to a row, 16 channels each
        // (4 at a time, 32 apart)
        const size_t block = run * NTILES + t;
        uint8_t* hp = a.h + block * C::X_BYTES;
#pragma unroll 1
        for (int i = et; i < (rows + 3) / 4 * 32; i += EPI) {
          const int n = i >> 3, l8 = i & 7;
          float v[16];
          float am = __uint_as_float(AMAX_MIN_BITS);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 w = n < rows ? *reinterpret_cast<const float4*>(hs + n * QB + 32 * j + 4 * l8) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * j] = w.x, v[4 * j + 1] = w.y, v[4 * j + 2] = w.z, v[4 * j + 3] = w.w;
            am = max_abs(max_abs(am, w.x, w.y), w.z, w.w);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) am = max_abs(am, __shfl_xor_sync(0xffffffffu, am, o), 0.f);
          if (n < rows) {
            const uint4 w = e4m3x16(v, BlockRatio(am));
            const uint32_t ws4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(hp + image_at(n, 32 * j + 4 * l8)) = ws4[j];
            if (l8 == 0) a.h_s[block * NT + n] = block_scale(am);
          }
        }
      }
      // (hs is written again after another barrier)
    }
    if (et == 0) *static_cast<volatile int*>(&ctl.over) = 1;
    if (owed) {  // given up
      hand_arrive<2>();
      handed = true;
    }
    if (handed) hand_sync<3>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <bool GATED, int NT, bool ROWS = false>
cudaError_t launch(const QGemmArgs& a, cudaStream_t st) {
  using C = Thin<GATED, NT>;
  const size_t smem = C::SMEM;
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(&k_qgemm_thin<GATED, NT, ROWS>), smem);
  if (e != cudaSuccess) return e;
  return launch_q(k_qgemm_thin<GATED, NT, ROWS>, dim3(a.num_sms), THREADS + (ROWS ? ROW_THREADS : 0) + HAND, smem, st, a,
                  ROWS ? *a.rows : QRowsArgs{});
}

}  // namespace

// Two slots per CTA of the widest kind of tile.
size_t qgemm_thin_parts(int num_sms, bool gated) { return static_cast<size_t>(2) * num_sms * 128 * 64 * (gated ? 2 : 1); }

cudaError_t launch_qgemm_thin(const QGemmArgs& a, bool gated, cudaStream_t st) {
  if (a.rows) return launch<false, 16, true>(a, st);
  if (gated) return a.G == 16 ? launch<true, 16>(a, st) : a.G == 32 ? launch<true, 32>(a, st) : launch<true, 64>(a, st);
  return a.G == 16 ? launch<false, 16>(a, st) : a.G == 32 ? launch<false, 32>(a, st) : launch<false, 64>(a, st);
}

}  // namespace pop
