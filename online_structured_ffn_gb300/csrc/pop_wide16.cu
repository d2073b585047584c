// Products of 16-bit operands on 256 x 256 tiles with fused epilogues (pop_wide16.h).
//
// Two CTAs of a cluster work as a pair on 256 rows by 256 columns (cta_group::2): each brings its own 128 rows and 128
// columns of a k-block of 64, 32 KB by TMA into a ring of six (8-bit: of four), and has its rows' 256 fp32 sums in tensor
// memory, twice, so that the epilogue of one tile runs under the products of the next. An operand with k contiguous is one box
// of 64 x 128; one with the other side contiguous two boxes of 64 values by 64 k, and the tensor cores read it mn-major,
// so no matrix is transposed in memory. Gate and up: the first CTA brings 128 rows of Wg, the second the same of W1, so
// columns 0..127 of a tile are the gates and 128..255 the ups of 128 channels. Tiles may be narrower (wide16_width), so
// that the last round of them is full.
//
// Many tiles go round the pairs. Few tiles of long sums are each given to a cluster of S pairs, which take a run of the k-blocks
// each; then every CTA sums 1 / S of the columns, the others' parts of them read from their shared memory, and has the
// epilogue of those alone. (Tiles of a last round shared through global memory, summed by the pair that came last, cost 25 us
// and more: 128 KB of each CTA's part written and read again, one CTA reading them all.)
//
// 8-bit integers (there is no tensor-core product of them on sm_103a): exact in fp16, the rows are kept so; the matrix comes as
// 8-bit blocks, which twelve more warps turn into fp16 operands in shared memory on the way.
//
// Bound by the tensor cores, of many rows by the power limit: gate and up of 2048 tokens by 2 x 11008 x 4096 188 us (1.96 PFLOP/s,
// tensor cores busy 95 %), down 98 (1.88; 92 %); gradients of the matrices of 1024 tokens 162 (1.71; 81 %, as their tiles have
// 16 k-blocks), of the hidden values 71, whose epilogue reads 6 bytes a value and writes 4 (69 %). A k-block of a pair takes
// 0.27 us; of 8-bit integers 0.30.
//
// Persistent, one CTA per SM. Warp 0: copies. Warp 1: of the first CTA the products of both, of the second the news that
// its operands have landed. Warps 4..11: epilogue, TMEM lane quarter warp % 4, half of the columns each. Every wait has a
// limit; a CTA that gives up records WERR_TIMEOUT, lets its copies and products finish, frees TMEM and returns.
#include "pop_wide16.h"

#include <atomic>

#include "pop_qdevice.cuh"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int BM = 128, BK = 64;
constexpr int MAX_STAGES = 6;
constexpr uint32_t A_BYTES = BM * BK * 2, STAGE = 2 * A_BYTES;
constexpr uint32_t BOX_MN = 64 * 64 * 2;  // one of an mn-major operand's two boxes
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t OUT_BYTES = 8 * 32 * 128;  // 128 bytes of 32 rows on their way out, of each epilogue warp
constexpr int RING8 = 6;                      // blocks of 128 rows by 64 k of 8-bit integers on their way
constexpr uint32_t BLOCK8 = W8_BLOCK;
constexpr int WIDEST = 256;                    // columns of a tile
constexpr int GROUP = 8;                      // row tiles that share the columns' passes

struct Ctl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t full8[RING8], empty8[RING8];
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

template <WKind KIND>
struct Kind {
  static constexpr bool gated = KIND == W_GATED || KIND == W_I8_GATED;
  static constexpr bool i8 = KIND == W_I8 || KIND == W_I8_GATED;
  static constexpr bool a_mn = KIND == W_DW;
  static constexpr bool b_mn = KIND == W_DGATED || KIND == W_DX || KIND == W_DW;
  static constexpr int segments = KIND == W_DX ? 2 : 1;
  static constexpr int threads = i8 ? 768 : 384;
  static constexpr int stages = i8 ? 4 : 6;
  static constexpr uint32_t ring = stages * STAGE + (i8 ? RING8 * BLOCK8 : 0);
};

// kind::f16 on both CTAs' tensor cores, a k-block (four products of 16). a_lo, b_lo: the descriptors' low words; a k-major
// operand's next 16 k are 32 bytes on, an mn-major one's 16 rows of 128 bytes.
template <bool A_MN, bool B_MN>
__device__ __forceinline__ void umma_pair16(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool first) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo + (A_MN ? 128 : 2) * k), "r"(b_lo + (B_MN ? 128 : 2) * k), "r"(idesc), "r"(DESC_HI),
        "r"(k > 0 || !first ? 1u : 0u)
        : "memory");
}
template <bool MN>
__device__ __forceinline__ uint32_t operand_lo(uint32_t saddr) {
  return ((saddr >> 4) & 0x3FFFu) | ((MN ? BOX_MN >> 4 : 1u) << 16);
}

struct Tile {
  int p, m, n;  // product, row tile, column tile
};

// Tiles in groups of GROUP row tiles, columns outermost within a group: neighbours, which run at the same time, share
// their rows' and their columns' operands in L2.
template <WKind KIND>
__device__ __forceinline__ Tile tile_at(const WArgs& a, int t) {
  const int cols = Kind<KIND>::gated ? a.width >> 1 : a.width;
  Tile r{0, 0, 0};
  int mt = qceil(a.m[0], 2 * BM), nt = qceil(a.n[0], cols);
  if (KIND == W_DW) {
#pragma unroll
    for (int p = 1; p < 3; ++p) {
      if (r.p != p - 1 || p >= a.problems || t < mt * nt) continue;
      t -= mt * nt;
      r.p = p;
      mt = qceil(a.m[p], 2 * BM);
      nt = qceil(a.n[p], cols);
    }
  }
  const int group = t / (GROUP * nt);
  const int rows = min(GROUP, mt - group * GROUP);
  t -= group * GROUP * nt;
  r.n = t / rows;
  r.m = group * GROUP + t - r.n * rows;
  return r;
}

// Arrives on `bar` in the CTAs of `mask` once all products issued so far by this thread have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t mask) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tcvt.u16.u32 m, %1;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(smem_u32(bar)),
      "r"(mask)
      : "memory");
}

using OutBuf = uint4 (*)[8];  // 32 rows of 128 bytes, a row's pieces of 16 in the order piece ^ (row % 8)

// A lane's 16 bytes of its row into the buffer, and 32 rows of up to 128 bytes out of it as whole lines. `limit`: bytes of a
// row that exist.
__device__ __forceinline__ void put(OutBuf buf, int lane, int piece, uint4 w) { buf[lane][piece ^ (lane & 7)] = w; }
__device__ __forceinline__ void flush_rows(OutBuf buf, int lane, uint8_t* y, size_t row_bytes, int rows, int limit) {
  __syncwarp();
  const int row = lane >> 3, piece = lane & 7;
  y += row * row_bytes + 16 * piece;
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    if (row + i < rows && 16 * piece < limit) *reinterpret_cast<uint4*>(y + i * row_bytes) = buf[row + i][piece ^ ((row + i) & 7)];
  __syncwarp();
}

// The same for 32 fp32 columns, added to what y holds where asked, to y in its type: four columns a lane and row.
__device__ __forceinline__ void flush_f32(OutBuf buf, int lane, void* y, size_t at, long long ldy, int rows, int cols, bool f32, bool add,
                                          bool even) {
  __syncwarp();
  const int piece = lane & 7, n = min(4, cols - 4 * piece);
#pragma unroll 1
  for (int row = lane >> 3; row < rows && n > 0; row += 4) {
    const uint4 w = buf[row][piece ^ (row & 7)];
    float f[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
    const size_t o = at + static_cast<size_t>(row) * ldy + 4 * piece;
    float* pf = static_cast<float*>(y) + o;
    uint16_t* ph = static_cast<uint16_t*>(y) + o;
    if (even && n == 4) {
      if (add && f32) {
        const float4 old = *reinterpret_cast<const float4*>(pf);
        f[0] += old.x, f[1] += old.y, f[2] += old.z, f[3] += old.w;
      } else if (add) {
        const uint2 old = *reinterpret_cast<const uint2*>(ph);
        f[0] += bf16lo(old.x), f[1] += bf16hi(old.x), f[2] += bf16lo(old.y), f[3] += bf16hi(old.y);
      }
      if (f32)
        *reinterpret_cast<float4*>(pf) = make_float4(f[0], f[1], f[2], f[3]);
      else
        *reinterpret_cast<uint2*>(ph) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= n) continue;
        if (f32)
          pf[j] = add ? pf[j] + f[j] : f[j];
        else
          ph[j] = static_cast<uint16_t>(pack_bf16x2(add ? f[j] + bf16lo(ph[j]) : f[j], 0.f));
      }
    }
  }
  __syncwarp();
}

// Sixteen columns of tensor memory as floats, and back.
__device__ __forceinline__ void columns16(uint32_t taddr, float* v) {
  uint32_t r[16];
  tmem_load(taddr, r);
  tmem_wait(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void columns32(uint32_t taddr, float* v) {
  uint32_t r[2][16];
  tmem_load(taddr, r[0]);
  tmem_load(taddr + 16, r[1]);
  tmem_wait(r[0]);
  tmem_wait(r[1]);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i >> 4][i & 15]);
}
__device__ __forceinline__ void set_columns16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
      "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

// Kept gate and up values of sixteen channels, [channel pair][3 words].
__device__ __forceinline__ void load_kept(const uint32_t* from, int c, int cols, uint32_t (&k)[24]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool is = c + 2 * j < cols;
#pragma unroll
    for (int i = 0; i < 3; ++i) k[3 * j + i] = is ? __ldcg(from + (c / 2 + j) * 96 + 32 * i) : 0u;
  }
}

template <WKind KIND>
__global__ void __launch_bounds__(Kind<KIND>::threads, 1) k_wide16(const __grid_constant__ WArgs a) {
  using T = Kind<KIND>;
  constexpr int STAGES = T::stages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl.abort_flag;
  const int in_cluster = static_cast<int>(cluster_rank()), S = static_cast<int>(cluster_ctas()) >> 1;
  const int rank = in_cluster & 1, part = in_cluster >> 1;  // within the pair; which run of the k-blocks
  const uint32_t leader_cta = in_cluster & ~1;
  const int tile0 = S == 1 ? blockIdx.x >> 1 : blockIdx.x / (2 * S), tile_step = S == 1 ? gridDim.x >> 1 : a.tiles;
  const int W2 = a.width >> 1, out_cols = T::gated ? W2 : a.width;  // columns of either CTA's B; outputs (channels) of a tile
  const int KB = a.kb * T::segments, kb0 = KB * part / S, kb1 = KB * (part + 1) / S;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      // its own operands (8-bit: and word of the four warps that convert B); the first CTA's: and word of the second's
      mbar_init(&ctl.full[s], (rank == 0 ? 2 : 1) + (T::i8 ? 4 : 0));
      mbar_init(&ctl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.tfull[b], 1);
      mbar_init(&ctl.tempty[b], 16);  // the first CTA's: the epilogue warps of both
    }
    for (int s = 0; s < RING8 && T::i8; ++s) {
      mbar_init(&ctl.full8[s], 1);
      mbar_init(&ctl.empty8[s], 4);
    }
    mbar_init(&ctl.drain, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&ctl.tmem_base, TMEM_COLS);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = ctl.tmem_base;

  auto fail = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      atomicOr(a.err, WERR_TIMEOUT);
    }
  };

  if (warp < 4) {
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- copies (one thread)
      uint32_t issued = 0, s = 0, phase = 1;
      bool ok = true;
      // The first stages' B goes out before the kernel before this one has ended, where that does not write it.
      int early = a.b_early && !T::i8 ? min(STAGES, kb1 - kb0) : 0;
      if (!early) pdl_wait();
      for (int t = tile0; t < a.tiles && ok; t += tile_step) {
        const Tile tile = tile_at<KIND>(a, t);
        const int m0 = tile.m * 2 * BM + rank * BM;
        // A CTA without rows multiplies what its stages hold, and nothing reads the products.
        const bool any = m0 < a.m[tile.p];
        const uint32_t b_bytes = T::i8 ? 0 : T::b_mn ? (W2 > 64 ? 2 : 1) * BOX_MN : W2 * BK * 2;
        const int n0 = T::gated ? tile.n * W2 : tile.n * a.width + rank * W2;
        const CUtensorMap* ma = &a.map[KIND == W_DW ? 2 * tile.p : 0];
        const CUtensorMap* mb = T::gated ? &a.map[1 + rank] : ma + 1;
        const auto load = [&](int i, int stage, bool left, bool right) {
          const bool second = KIND == W_DX && i >= a.kb;
          const int x = (second ? i - a.kb : i) * BK;
          const CUtensorMap *pa = ma + (second ? 2 : 0), *pb = mb + (second ? 2 : 0);
          uint8_t* st = smem + stage * STAGE;
          uint64_t* bar = &ctl.full[stage];
          if (left && T::a_mn) {
            tma_load_2d(st, pa, bar, m0, x);
            tma_load_2d(st + BOX_MN, pa, bar, m0 + 64, x);
          } else if (left) {
            tma_load_2d(st, pa, bar, x, m0);
          }
          if (right && T::b_mn) {
            tma_load_2d(st + A_BYTES, pb, bar, n0, x);
            if (W2 > 64) tma_load_2d(st + A_BYTES + BOX_MN, pb, bar, n0 + 64, x);
          } else if (right && !T::i8) {
            tma_load_2d(st + A_BYTES, pb, bar, x, n0);
          }
        };
        const uint32_t bytes = (any ? A_BYTES : 0) + b_bytes;
        if (early) {
          for (int i = 0; i < early; ++i) {
            mbar_arrive_expect_tx(&ctl.full[i], bytes);
            load(kb0 + i, i, false, true);
          }
          pdl_wait();
        }
        for (int i = kb0; i < kb1; ++i) {
          if (!mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          if (!early) mbar_arrive_expect_tx(&ctl.full[s], bytes);
          load(i, s, any, !early);
          if (early) --early;
          ++issued;
          if (++s == STAGES) s = 0, phase ^= 1;
        }
      }
      // No copy of this CTA may be in flight when it exits. (The first CTA's barriers also wait for word of the second,
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
    if (T::i8 && warp == 2 && lane == 0) {
      // ---------------------------------------------------------- 8-bit blocks of the matrix (one thread)
      uint32_t issued = 0, s = 0, phase = 1;
      bool ok = true;
      for (int t = tile0; t < a.tiles && ok; t += tile_step) {
        const Tile tile = tile_at<KIND>(a, t);
        const int last = qceil(a.n[0], 128) - 1;  // (a tile past it is not looked at)
        const uint8_t* w = a.w8[T::gated ? rank : 0] +
                           (static_cast<size_t>(T::gated ? tile.n : min(2 * tile.n + rank, last)) * KB + kb0) * BLOCK8;
        for (int i = kb0; i < kb1; ++i, w += BLOCK8) {
          if (!mbar_wait(&ctl.empty8[s], phase, a.wait, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&ctl.full8[s], BLOCK8);
          bulk_load(smem + STAGES * STAGE + s * BLOCK8, w, BLOCK8, &ctl.full8[s]);
          ++issued;
          if (++s == RING8) s = 0, phase ^= 1;
        }
      }
      const uint32_t lo = issued > RING8 ? issued - RING8 : 0;
      for (uint32_t i = lo; i < issued; ++i) {
        volatile int never = 0;
        if (!mbar_wait(&ctl.full8[i % RING8], (i / RING8) & 1u, Q_DRAIN, &never)) {
          fail();
          break;
        }
      }
    }
    if (warp == 1) {
      const bool leader = elect_one();
      uint32_t s = 0, phase = 0, b = 0, tphase = 1;
      if (rank == 0) {
        // -------------------------------------------------------- products
        const uint32_t idesc = idesc_bf16_f32(2 * BM, a.width, T::b_mn, T::a_mn) & ~(T::i8 ? (1u << 7) | (1u << 10) : 0u);
        const uint32_t a0 = operand_lo<T::a_mn>(smem_u32(smem)), b0 = operand_lo<T::b_mn>(smem_u32(smem) + A_BYTES);
        const uint32_t mask = 3u << leader_cta;
        bool ok = true;
        for (int t = tile0; t < a.tiles && ok; t += tile_step) {
          if (!mbar_wait(&ctl.tempty[b], tphase, a.wait, abort_flag)) {
            if (leader) fail();
            break;
          }
          tc_fence_after();
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&ctl.full[s], phase, a.wait, abort_flag)) {
              if (leader) fail();
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) {
              umma_pair16<T::a_mn, T::b_mn>(tmem_base + b * 256u, a0 + s * (STAGE >> 4), b0 + s * (STAGE >> 4), idesc, kb == kb0);
              commit_pair(&ctl.empty[s], mask);
              if (kb == kb1 - 1) commit_pair(&ctl.tfull[b], mask);
            }
            __syncwarp();
            if (++s == STAGES) s = 0, phase ^= 1;
          }
          b ^= 1u;
          tphase ^= b ^ 1u;
        }
        if (leader) commit_pair(&ctl.drain, mask);
        volatile int never = 0;
        if (!mbar_wait(&ctl.drain, 0, Q_DRAIN, &never) && leader) fail();
      } else {
        // -------------------------------------------------------- word of this CTA's operands
        const uint32_t first0 = in_cta(&ctl.full[0], leader_cta);
        bool ok = true;
        for (int t = tile0; t < a.tiles && ok; t += tile_step) {
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&ctl.full[s], phase, a.wait, abort_flag)) {
              if (leader) fail();
              ok = false;
              break;
            }
            if (leader) mbar_arrive_first(first0 + s * 8u);
            __syncwarp();
            if (++s == STAGES) s = 0, phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (T::i8 && warp >= 12) {
    // ------------------------------------------------------------ 8-bit integers to fp16 (warps 12..23)
    // A row each thread, every third k-block the same four warps: a block takes a warp longer than its products take (with one set
    // of warps 0.36 us and more a k-block, two 0.32, three 0.30; at the power limit, 4001 x 28672 x 8192, three are 2 % behind two).
    // A slot of the ring has the same four every time: others, who have not looked at it before, could not tell a block that has
    // not landed from the one before it, and copies may land out of order. (Stages are freed in order.)
    constexpr int SETS = 3;
    static_assert(RING8 % SETS == 0 && (!T::i8 || T::threads == 384 + 128 * SETS), "a slot's warps");
    const int r = threadIdx.x & 127;
    int left = -((warp - 12) >> 2);  // blocks of this CTA
    for (int t = tile0; t < a.tiles; t += tile_step) left += kb1 - kb0;
    uint32_t s = (warp - 12) >> 2, phase = 1, s8 = s, phase8 = 0;
    for (; left > 0; left -= SETS) {
      const bool ok = mbar_wait(&ctl.full8[s8], phase8, a.wait, abort_flag) && mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) fail();
        break;
      }
      const uint4* from = reinterpret_cast<const uint4*>(smem + STAGES * STAGE + s8 * BLOCK8) + r;
      uint8_t* to = smem + s * STAGE + A_BYTES + r * 128;
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = from[128 * j];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<uint4*>(to + (((2 * j) ^ (r & 7)) << 4)) = half8(v[j].x, v[j].y);
        *reinterpret_cast<uint4*>(to + (((2 * j + 1) ^ (r & 7)) << 4)) = half8(v[j].z, v[j].w);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.full[s]);
        mbar_arrive(&ctl.empty8[s8]);
      }
      s += SETS;
      if (s >= STAGES) s -= STAGES, phase ^= 1;
      s8 += SETS;
      if (s8 >= RING8) s8 -= RING8, phase8 ^= 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (warps 4..11)
    pdl_wait();  // what this kernel writes may still be read by the one before
    pdl_trigger();
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    const uint32_t tempty0 = in_cta(&ctl.tempty[0], leader_cta), tempty1 = in_cta(&ctl.tempty[1], leader_cta);
    OutBuf buf = reinterpret_cast<OutBuf>(smem + T::ring + (warp - 4) * (32 * 128));
    uint32_t b = 0, tphase = 0;
    // Once a wait has run out the rest is gone through without waiting or storing, and nobody is told that a buffer has been
    // read.
    bool ok = true;
    for (int t = tile0; t < a.tiles; t += tile_step) {
      const Tile tile = tile_at<KIND>(a, t);
      const int M = a.m[tile.p], N = a.n[tile.p];
      const int row0 = tile.m * 2 * BM + rank * BM + 32 * q;  // this warp's first row
      const int rows = min(32, M - row0);                     // may be none
      // outputs of this CTA (of three, whole pieces of 32), and of its warps of the lower half
      const int first = S == 1 ? 0 : (out_cols * part / S) & ~31, end = S == 1 ? out_cols : (out_cols * (part + 1) / S) & ~31;
      const int lower = ((end - first) / 2 + 15) & ~15, wide = half ? end - first - lower : lower;
      const int at0 = first + (half ? lower : 0);             // this warp's first one within the tile
      const int col0 = tile.n * out_cols + at0;
      const int cols = min(wide, N - col0);                   // may be none
      const bool some = rows > 0 && cols > 0;
      const uint32_t* from = KIND == W_DGATED ? a.saved + (static_cast<size_t>(row0 >> 5) * (N >> 1) + (col0 >> 1)) * 96 + lane : nullptr;
      uint32_t k0[24], k1[24];
      if (KIND == W_DGATED && some) {
        load_kept(from, 0, cols, k0);
        load_kept(from, 16, cols, k1);
      }
      ok = ok && mbar_wait(&ctl.tfull[b], tphase, a.wait, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok && lane == 0) fail();
      tc_fence_after();
      const uint32_t taddr = lane_base + b * 256u + at0;  // gated: the ups are W2 further on
      if (S > 1) {
        // What the others are to sum goes to shared memory, where the products no longer read: [column / 4][row][4].
        float4* mine = reinterpret_cast<float4*>(smem) + 32 * q + lane;
        if (ok && rows > 0) {
#pragma unroll 1
          for (int c = 128 * half; c < 128 * half + 128; c += 32) {
            const int o = T::gated ? c & 127 : c;
            if (o >= first && o < end) continue;
            float f[32];
            columns32(lane_base + c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) mine[(c / 4 + j) * BM] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
          }
        }
        cluster_sync();
        // The parts in the order of k, this CTA's own from tensor memory, where the sums go.
        if (ok && some) {
#pragma unroll 1
          for (int c = 0; c < (T::gated ? 2 * wide : wide); c += 16) {
            // gated: the gates, then as many ups
            const int col = at0 + (T::gated && c >= wide ? 128 - wide : 0) + c;
            float f[16], keep[16];
            columns16(lane_base + col, keep);
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = 0.f;
#pragma unroll 1
            for (int p = 0; p < S; ++p) {
              if (p == part) {
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] += keep[j];
                continue;
              }
              const uint32_t from = in_cta(mine + col / 4 * BM, 2 * p + rank);
              float4 x[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = ld_cluster(from + j * BM * 16);
#pragma unroll
              for (int j = 0; j < 4; ++j) f[4 * j] += x[j].x, f[4 * j + 1] += x[j].y, f[4 * j + 2] += x[j].z, f[4 * j + 3] += x[j].w;
            }
            set_columns16(lane_base + col, f);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
      }
      // (Rolled loops: as straight-line code the largest of these epilogues was some 80 KB, and fetching it took longer
      // than running it: a tile's 27 us.)
      if (ok && some) {
        if (KIND == W_GATED) {
          uint32_t* keep = a.saved ? a.saved + (static_cast<size_t>(row0 >> 5) * (N >> 1) + (col0 >> 1)) * 96 + lane : nullptr;
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            float g[16], u[16];
            columns16(taddr + c, g);
            columns16(taddr + W2 + c, u);
            uint32_t p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = pack_bf16x2(silu_mul(g[2 * j], u[2 * j]), silu_mul(g[2 * j + 1], u[2 * j + 1]));
            put(buf, lane, c / 8, make_uint4(p[0], p[1], p[2], p[3]));
            put(buf, lane, c / 8 + 1, make_uint4(p[4], p[5], p[6], p[7]));
            if (keep) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                if (c + 2 * j >= cols) break;
                const uint32_t g0 = __float_as_uint(g[2 * j]), g1 = __float_as_uint(g[2 * j + 1]);
                const uint32_t u0 = __float_as_uint(u[2 * j]), u1 = __float_as_uint(u[2 * j + 1]);
                uint32_t* k = keep + (c / 2 + j) * 96;
                __stcg(k, __byte_perm(g0, g1, 0x7632));
                __stcg(k + 32, __byte_perm(u0, u1, 0x7632));
                __stcg(k + 64, __byte_perm(__byte_perm(g0, g1, 0x0051), __byte_perm(u0, u1, 0x0051), 0x5410));
              }
            }
          }
          flush_rows(buf, lane, reinterpret_cast<uint8_t*>(a.h) + (static_cast<size_t>(row0) * N + col0) * 2, static_cast<size_t>(N) * 2,
                     rows, 2 * cols);
        } else if (KIND == W_I8_GATED) {
          const float sx = lane < rows ? a.sx[row0 + lane] : 0.f;
          float most = 0.f;
#pragma unroll 1
          for (int c = 0; c < cols; c += 32) {
#pragma unroll 1
            for (int i = 0; i < 32; i += 16) {
              float g[16], u[16];
              columns16(taddr + c + i, g);
              columns16(taddr + W2 + c + i, u);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int ch = min(col0 + c + i + j, N - 1);
                g[j] = silu_mul(g[j] * (sx * __ldg(a.sw + ch)), u[j] * (sx * __ldg(a.sw1 + ch)));
                if (c + i + j < cols) most = max_abs(most, g[j], 0.f);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                put(buf, lane, i / 4 + j, make_uint4(__float_as_uint(g[4 * j]), __float_as_uint(g[4 * j + 1]), __float_as_uint(g[4 * j + 2]),
                                                     __float_as_uint(g[4 * j + 3])));
            }
            flush_f32(buf, lane, a.hf, static_cast<size_t>(row0) * N + col0 + c, N, rows, cols - c, true, false, true);
          }
          if (lane < rows) atomicMax(a.amax + row0 + lane, __float_as_uint(most));
        } else if (KIND == W_DGATED) {
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            uint32_t k[24];
#pragma unroll
            for (int j = 0; j < 24; ++j) k[j] = k0[j], k0[j] = k1[j];
            load_kept(from, c + 32, cols, k1);  // two chunks ahead
            float dh[16];
            columns16(taddr + c, dh);
            uint32_t dg[8], du[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float o[2][2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // (the lowest byte repeats the one above it: less than the bits that were not kept)
                const float g = __uint_as_float(__byte_perm(k[3 * j], k[3 * j + 2], i ? 0x3255 : 0x1044));
                const float u = __uint_as_float(__byte_perm(k[3 * j + 1], k[3 * j + 2], i ? 0x3277 : 0x1066));
                const float p = sigmoid(g), d = dh[2 * j + i];
                o[0][i] = d * u * (p * fmaf(g, 1.f - p, 1.f));
                o[1][i] = d * (g * p);
              }
              dg[j] = pack_bf16x2(o[0][0], o[0][1]);
              du[j] = pack_bf16x2(o[1][0], o[1][1]);
            }
            // 32 channels at a time: the gate's gradients, then the ups'
            const int at = (c >> 3) & 2;
            put(buf, lane, at, make_uint4(dg[0], dg[1], dg[2], dg[3]));
            put(buf, lane, at + 1, make_uint4(dg[4], dg[5], dg[6], dg[7]));
            put(buf, lane, at + 4, make_uint4(du[0], du[1], du[2], du[3]));
            put(buf, lane, at + 5, make_uint4(du[4], du[5], du[6], du[7]));
            if (at || c + 16 >= cols) {
              const int ch = c & ~31, row = lane >> 3, piece = lane & 7;
              __syncwarp();
              uint16_t* o = (piece < 4 ? a.h : a.h2) + static_cast<size_t>(row0 + row) * N + col0 + ch + 8 * (piece & 3);
              const bool is = ch + 8 * (piece & 3) < cols;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                if (row + i < rows && is) *reinterpret_cast<uint4*>(o + static_cast<size_t>(i) * N) = buf[row + i][piece ^ ((row + i) & 7)];
              __syncwarp();
            }
          }
        } else {
          const long long ldy = a.ldy[tile.p];
          void* y = a.y[tile.p];
          const int size = a.out_f32 ? 4 : 2;
          const bool even = KIND != W_I8 || (ldy * size % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0);
          const bool direct = !a.out_f32 && !a.accumulate && even && (KIND != W_I8 || N % 8 == 0);
          const float sx = KIND == W_I8 && lane < rows ? a.sx[row0 + lane] : 0.f;
#pragma unroll 1
          for (int c = 0; c < cols; c += 16) {
            float f[16];
            columns16(taddr + c, f);
            if (KIND == W_I8) {
#pragma unroll
              for (int j = 0; j < 16; ++j) f[j] *= sx * __ldg(a.sw + min(col0 + c + j, N - 1));
            }
            if (direct) {
#pragma unroll
              for (int j = 0; j < 2; ++j)
                put(buf, lane, ((c >> 3) & 7) + j, make_uint4(pack_bf16x2(f[8 * j], f[8 * j + 1]), pack_bf16x2(f[8 * j + 2], f[8 * j + 3]),
                                                              pack_bf16x2(f[8 * j + 4], f[8 * j + 5]), pack_bf16x2(f[8 * j + 6], f[8 * j + 7])));
              if ((c & 48) == 48 || c + 16 >= cols)
                flush_rows(buf, lane, static_cast<uint8_t*>(y) + (static_cast<size_t>(row0) * ldy + col0 + (c & ~63)) * 2, ldy * 2, rows,
                           2 * (cols - (c & ~63)));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                put(buf, lane, ((c >> 2) & 7) + j, make_uint4(__float_as_uint(f[4 * j]), __float_as_uint(f[4 * j + 1]), __float_as_uint(f[4 * j + 2]),
                                                              __float_as_uint(f[4 * j + 3])));
              if ((c & 16) || c + 16 >= cols)
                flush_f32(buf, lane, y, static_cast<size_t>(row0) * ldy + col0 + (c & ~31), ldy, rows, cols - (c & ~31), a.out_f32, a.accumulate,
                          even);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive_first(b ? tempty1 : tempty0);
      b ^= 1u;
      tphase ^= b ^ 1u;
    }
  }

  if (S > 1 && (warp < 4 || warp >= 12)) cluster_sync();  // the others' exchange
  tc_fence_before();
  cluster_sync();  // nothing of any CTA is still used by another
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// Clusters of 2 S CTAs that the device holds at a time; asked once per kernel and device.
template <WKind KIND>
int clusters_at_a_time(int S, size_t smem, int num_sms) {
  static std::atomic<int> known[64][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& k = known[dev][S - 2];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(2 * S), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / (2 * S) * 2 * S);
    cfg.blockDim = dim3(Kind<KIND>::threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, k_wide16<KIND>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    n = n > 0 ? n : -1;
    k.store(n, std::memory_order_relaxed);
  }
  return n > 0 ? n : 0;
}

template <WKind KIND>
cudaError_t launch(WArgs a, cudaStream_t st) {
  const size_t smem = Kind<KIND>::ring + OUT_BYTES + 1024;
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(&k_wide16<KIND>), smem);
  if (e != cudaSuccess) return e;
  long long tiles = 0;
  for (int p = 0; p < (KIND == W_DW ? a.problems : 1); ++p)
    tiles += static_cast<long long>(qceil(a.m[p], 2 * BM)) * qceil(a.n[p], Kind<KIND>::gated ? a.width / 2 : a.width);
  if (tiles > (1 << 28)) return cudaErrorInvalidValue;
  a.tiles = static_cast<int>(tiles);
  const int KB = a.kb * Kind<KIND>::segments, pairs = a.num_sms / 2;
  // As many pairs to a tile as there are for all tiles at once, with two k-blocks each at least, of three with sixteen. (200 rows
  // by 2 x 11008 x 4096 and back, whose second product has 16 tiles of 172: 64 us with 3, 69 with 2; gate and up by 2 x 2736 x 1000, 22
  // tiles of 16: 2.3 us more.)
  // The gradients of the matrices go by the tiles of all three, whichever are asked for, as S is how a gradient's sum is split: what
  // else is wanted is not to change its bits. (All three have as many tiles. That of W2 alone, with S by its own tiles and by all
  // of them: 512 x 512 x 1024 9.1 and 7.4 us, 600 x 264 x 1032 9.3 and 8.1, 1000 x 264 x 2056 9.2 and 10.2, 2048 x 1024 x 1024 10.7 and
  // 12.9.)
  const long long sharing = KIND == W_DW ? 3ll * qceil(a.m[0], 2 * BM) * qceil(a.n[0], a.width) : tiles;
  int S = 1;
  for (int s = 4; s > 1 && S == 1; --s)
    if (a.width == WIDEST && sharing * s <= pairs && KB >= (s == 3 ? 48 : 2 * s) && sharing <= clusters_at_a_time<KIND>(s, smem, a.num_sms)) S = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(2 * S), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * S * (a.tiles < pairs ? a.tiles : pairs));
  cfg.blockDim = dim3(Kind<KIND>::threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_wide16<KIND>, a);
}

}  // namespace

// The width for which the rounds of tiles over the pairs take least. Where the widest tiles leave half the pairs idle those are
// shared instead. A round takes its columns' time, and that of some 24 more. An mn-major B's boxes do not get narrower
// with the tile, so there it takes that of 350 more, and widths between whole pieces of 32 columns are slower still. 8-bit
// matrices come in blocks of 128 rows. (Forward of 4096 x 4096 x 11008 in us, at 256 columns 646, 240 617, 224 567, 208 595, 192
// 615, 160 656; of 1000 rows 156, 153, 157, 187, 191, 195. Gradients of x and the hidden values, 4096 rows 645, 765, 628, 812,
// 728, 800; 777 x 2048 x 5496 65, 112, 89, 110, 88, 87, and 62 with 160 columns for the hidden ones alone.)
int wide16_width(WKind kind, int m, int n, int num_sms) {
  const int pairs = num_sms / 2;
  const bool gated = kind == W_GATED, mn = kind == W_DGATED || kind == W_DX;
  const long long mt = qceil(m, 2 * BM);
  if (kind == W_I8 || kind == W_I8_GATED || kind == W_DW || mt * qceil(n, gated ? WIDEST / 2 : WIDEST) * 2 <= pairs) return WIDEST;
  int best = WIDEST;
  long long least = -1;
  for (int w = WIDEST; w >= 128; w -= mn ? 32 : 16) {
    const long long rounds = (mt * qceil(n, gated ? w / 2 : w) + pairs - 1) / pairs, cost = rounds * (w + (mn ? 350 : 24));
    if (least < 0 || cost < least) least = cost, best = w;
  }
  return best;
}

cudaError_t launch_wide16(WKind kind, const WArgs& a, cudaStream_t st) {
  switch (kind) {
    case W_GATED: return launch<W_GATED>(a, st);
    case W_PLAIN: return launch<W_PLAIN>(a, st);
    case W_DGATED: return launch<W_DGATED>(a, st);
    case W_DX: return launch<W_DX>(a, st);
    case W_DW: return launch<W_DW>(a, st);
    case W_I8: return launch<W_I8>(a, st);
    case W_I8_GATED: return launch<W_I8_GATED>(a, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rows16(WKind kind, WArgs a, cudaStream_t st) {
  if (a.m[0] <= THIN16_MOST) return launch_thin16(kind, a, st);
  if (!a.width) a.width = wide16_width(kind, a.m[0], a.n[0], a.num_sms);
  for (int i = 0; i < (kind == W_DX ? 2 : 1); ++i)
    if (!encode_map16(&a.map[2 * i], i ? a.rows2 : a.rows, a.k, a.m[0], static_cast<uint64_t>(a.ld_rows) * 2, BK, BM))
      return cudaErrorInvalidValue;
  return launch_wide16(kind, a, st);
}

}  // namespace pop
