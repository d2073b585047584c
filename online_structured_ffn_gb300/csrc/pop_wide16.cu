// Products of 16-bit operands on 256 x 256 tiles with fused epilogues (pop_wide16.h).
//
// Two CTAs of a cluster work as a pair on 256 rows by 256 columns (cta_group::2): each brings its own 128 rows and 128
// columns of a k-block of 64, 32 KB by TMA into a ring of six, and has its rows' 256 fp32 sums in tensor memory, twice, so
// that the epilogue of one tile runs under the products of the next. An operand with k contiguous is one box of
// 64 x 128; one with the other side contiguous two boxes of 64 values by 64 k, and the tensor cores read it mn-major, so
// no matrix is transposed in memory. Gate and up: the first CTA brings 128 rows of Wg, the second the same of W1,
// so columns 0..127 of a tile are the gates and 128..255 the ups of 128 channels.
//
// Persistent, one CTA per SM. Warp 0: copies. Warp 1: of the first CTA the products of both, of the second the news that
// its operands have landed. Warps 4..11: epilogue, TMEM lane quarter warp % 4, half of the columns each. Every wait has a
// limit; a CTA that gives up records WERR_TIMEOUT, lets its copies and products finish, frees TMEM and returns.
#include "pop_wide16.h"

#include "pop_qdevice.cuh"

namespace pop {

cudaError_t ensure_dyn_smem(const void* kernel, size_t bytes);

namespace {

constexpr int THREADS = 384;
constexpr int BM = 128, BK = 64;
constexpr int STAGES = 6;
constexpr uint32_t A_BYTES = BM * BK * 2, STAGE = 2 * A_BYTES;
constexpr uint32_t BOX_MN = 64 * 64 * 2;  // one of an mn-major operand's two boxes
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t OUT_BYTES = 8 * 32 * 128;  // 128 bytes of 32 rows on their way out, of each epilogue warp
constexpr int GROUP = 8;                      // row tiles that share the columns' passes

struct Ctl {
  uint64_t full[STAGES], empty[STAGES];
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
  static constexpr int cols = gated ? 128 : 256;  // outputs (channels) of a tile
  static constexpr int segments = KIND == W_DX ? 2 : 1;
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
  Tile r{0, 0, 0};
  int mt = qceil(a.m[0], 2 * BM), nt = qceil(a.n[0], Kind<KIND>::cols);
  if (KIND == W_DW) {
#pragma unroll
    for (int p = 1; p < 3; ++p) {
      if (r.p != p - 1 || p >= a.problems || t < mt * nt) continue;
      t -= mt * nt;
      r.p = p;
      mt = qceil(a.m[p], 2 * BM);
      nt = qceil(a.n[p], Kind<KIND>::cols);
    }
  }
  const int group = t / (GROUP * nt);
  const int rows = min(GROUP, mt - group * GROUP);
  t -= group * GROUP * nt;
  r.n = t / rows;
  r.m = group * GROUP + t - r.n * rows;
  return r;
}
template <WKind KIND>
__device__ __forceinline__ int tile_count(const WArgs& a) {
  int n = 0;
  for (int p = 0; p < (KIND == W_DW ? a.problems : 1); ++p) n += qceil(a.m[p], 2 * BM) * qceil(a.n[p], Kind<KIND>::cols);
  return n;
}

// sigma(g). __expf and __fdividef are off by a few units of 2^-23; what comes of them is rounded to bf16 or int8.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

using OutBuf = uint4 (*)[8];  // 32 rows of 128 bytes, a row's pieces of 16 in the order piece ^ (row % 8)

// 32 rows of 128 bytes from the warp's lanes, a row each, out as whole lines. `limit`: bytes of a row that exist.
__device__ __forceinline__ void put_rows(OutBuf buf, int lane, const uint4 (&w)[8], uint8_t* y, size_t row_bytes, int rows, int limit) {
#pragma unroll
  for (int i = 0; i < 8; ++i) buf[lane][i ^ (lane & 7)] = w[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 4 * i + (lane >> 3), piece = lane & 7;
    if (row < rows && 16 * piece < limit) *reinterpret_cast<uint4*>(y + row * row_bytes + 16 * piece) = buf[row][piece ^ (row & 7)];
  }
  __syncwarp();
}

// 32 fp32 columns of 32 rows, added to what y holds where asked, to y in its type: four columns a lane and row.
__device__ __forceinline__ void put_f32(OutBuf buf, int lane, const float (&v)[32], void* y, size_t at, long long ldy, int rows, int cols,
                                        bool f32, bool add, bool even) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    buf[lane][i ^ (lane & 7)] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                           __float_as_uint(v[4 * i + 3]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 4 * i + (lane >> 3), piece = lane & 7, n = min(4, cols - 4 * piece);
    if (row >= rows || n <= 0) continue;
    const uint4 w = buf[row][piece ^ (row & 7)];
    float f[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
    const size_t o = at + static_cast<size_t>(row) * ldy + 4 * piece;
    if (f32) {
      float* p = static_cast<float*>(y) + o;
      if (even && n == 4) {
        float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
        if (add) old = *reinterpret_cast<const float4*>(p);
        *reinterpret_cast<float4*>(p) = make_float4(f[0] + old.x, f[1] + old.y, f[2] + old.z, f[3] + old.w);
      } else {
        for (int j = 0; j < n; ++j) p[j] = add ? p[j] + f[j] : f[j];
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(y) + o;
      if (even && n == 4) {
        if (add) {
          const uint2 old = *reinterpret_cast<const uint2*>(p);
          f[0] += bf16lo(old.x), f[1] += bf16hi(old.x), f[2] += bf16lo(old.y), f[3] += bf16hi(old.y);
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
      } else {
        for (int j = 0; j < n; ++j) p[j] = static_cast<uint16_t>(pack_bf16x2(add ? f[j] + bf16lo(p[j]) : f[j], 0.f));
      }
    }
  }
  __syncwarp();
}

// Sixteen columns of tensor memory as floats.
__device__ __forceinline__ void columns16(uint32_t taddr, float* v) {
  uint32_t r[16];
  tmem_load(taddr, r);
  tmem_wait(r);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <WKind KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) k_wide16(const __grid_constant__ WArgs a) {
  using T = Kind<KIND>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl.abort_flag;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = tile_count<KIND>(a);
  const int KB = a.kb * T::segments;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl.full[s], rank == 0 ? 2 : 1);  // the first CTA's: its own operands, and word of the second's
      mbar_init(&ctl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl.tfull[b], 1);
      mbar_init(&ctl.tempty[b], 16);  // the first CTA's: the epilogue warps of both
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
      pdl_wait();
      for (int t = pair; t < tiles && ok; t += pairs) {
        const Tile tile = tile_at<KIND>(a, t);
        const int m0 = tile.m * 2 * BM + rank * BM;
        const int n0 = T::gated ? tile.n * 128 : tile.n * 256 + rank * BM;
        const CUtensorMap* ma = &a.map[KIND == W_DW ? 2 * tile.p : 0];
        const CUtensorMap* mb = T::gated ? &a.map[1 + rank] : ma + 1;
        int kb = 0;
        for (int i = 0; i < KB; ++i, ++kb) {
          if (KIND == W_DX && i == a.kb) {
            ma += 2;
            mb += 2;
            kb = 0;
          }
          if (!mbar_wait(&ctl.empty[s], phase, a.wait, abort_flag)) {
            fail();
            ok = false;
            break;
          }
          uint8_t* st = smem + s * STAGE;
          mbar_arrive_expect_tx(&ctl.full[s], STAGE);
          if (T::a_mn) {
            tma_load_2d(st, ma, &ctl.full[s], m0, kb * BK);
            tma_load_2d(st + BOX_MN, ma, &ctl.full[s], m0 + 64, kb * BK);
          } else {
            tma_load_2d(st, ma, &ctl.full[s], kb * BK, m0);
          }
          if (T::b_mn) {
            tma_load_2d(st + A_BYTES, mb, &ctl.full[s], n0, kb * BK);
            tma_load_2d(st + A_BYTES + BOX_MN, mb, &ctl.full[s], n0 + 64, kb * BK);
          } else {
            tma_load_2d(st + A_BYTES, mb, &ctl.full[s], kb * BK, n0);
          }
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
    if (warp == 1) {
      const bool leader = elect_one();
      uint32_t s = 0, phase = 0, b = 0, tphase = 1;
      if (rank == 0) {
        // -------------------------------------------------------- products
        constexpr uint32_t IDESC = idesc_bf16_f32(2 * BM, 256, T::b_mn, T::a_mn) & ~(T::i8 ? (1u << 7) | (1u << 10) : 0u);
        const uint32_t a0 = operand_lo<T::a_mn>(smem_u32(smem)), b0 = operand_lo<T::b_mn>(smem_u32(smem) + A_BYTES);
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
          if (!mbar_wait(&ctl.tempty[b], tphase, a.wait, abort_flag)) {
            if (leader) fail();
            break;
          }
          tc_fence_after();
          for (int kb = 0; kb < KB; ++kb) {
            if (!mbar_wait(&ctl.full[s], phase, a.wait, abort_flag)) {
              if (leader) fail();
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) {
              umma_pair16<T::a_mn, T::b_mn>(tmem_base + b * 256u, a0 + s * (STAGE >> 4), b0 + s * (STAGE >> 4), IDESC, kb == 0);
              umma_commit_pair(&ctl.empty[s]);
              if (kb == KB - 1) umma_commit_pair(&ctl.tfull[b]);
            }
            __syncwarp();
            if (++s == STAGES) s = 0, phase ^= 1;
          }
          b ^= 1u;
          tphase ^= b ^ 1u;
        }
        if (leader) umma_commit_pair(&ctl.drain);
        volatile int never = 0;
        if (!mbar_wait(&ctl.drain, 0, Q_DRAIN, &never) && leader) fail();
      } else {
        // -------------------------------------------------------- word of this CTA's operands
        const uint32_t first0 = first_cta(&ctl.full[0]);
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs) {
          for (int kb = 0; kb < KB; ++kb) {
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
  } else {
    // ------------------------------------------------------------ epilogue (warps 4..11)
    pdl_wait();  // what this kernel writes may still be read by the one before
    pdl_trigger();
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    const uint32_t tempty0 = first_cta(&ctl.tempty[0]), tempty1 = first_cta(&ctl.tempty[1]);
    OutBuf buf = reinterpret_cast<OutBuf>(smem + STAGES * STAGE + (warp - 4) * (32 * 128));
    uint32_t b = 0, tphase = 0;
    for (int t = pair; t < tiles; t += pairs) {
      const Tile tile = tile_at<KIND>(a, t);
      const int M = a.m[tile.p], N = a.n[tile.p];
      const int row0 = tile.m * 2 * BM + rank * BM + 32 * q;  // this warp's first row
      const int rows = min(32, M - row0);                     // may be none
      if (!mbar_wait(&ctl.tfull[b], tphase, a.wait, abort_flag)) {
        if (lane == 0) fail();
        break;
      }
      __syncwarp();
      tc_fence_after();
      const uint32_t taddr = lane_base + b * 256u;
      if (KIND == W_GATED || KIND == W_I8_GATED) {
        const int ch0 = tile.n * 128 + 64 * half;
        const int cols = min(64, N - ch0);
        if (rows > 0 && cols > 0) {
          if (KIND == W_GATED) {
            uint32_t* keep = a.saved ? a.saved + (static_cast<size_t>(row0 >> 5) * (N >> 1) + (ch0 >> 1)) * 96 + lane : nullptr;
            uint4 w[8];
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
              float g[16], u[16];
              columns16(taddr + 64 * half + c, g);
              columns16(taddr + 128 + 64 * half + c, u);
              uint32_t p[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float h0 = silu_mul(g[2 * j], u[2 * j]), h1 = silu_mul(g[2 * j + 1], u[2 * j + 1]);
                p[j] = pack_bf16x2(h0, h1);
              }
              w[c / 8] = make_uint4(p[0], p[1], p[2], p[3]);
              w[c / 8 + 1] = make_uint4(p[4], p[5], p[6], p[7]);
              if (keep && c < cols) {  // (cols is a multiple of 8)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  if (c + 2 * j >= cols) break;
                  const uint32_t g0 = __float_as_uint(g[2 * j]), g1 = __float_as_uint(g[2 * j + 1]);
                  const uint32_t u0 = __float_as_uint(u[2 * j]), u1 = __float_as_uint(u[2 * j + 1]);
                  uint32_t* k = keep + (c / 2 + j) * 96;
                  __stcs(k, __byte_perm(g0, g1, 0x7632));
                  __stcs(k + 32, __byte_perm(u0, u1, 0x7632));
                  __stcs(k + 64, __byte_perm(__byte_perm(g0, g1, 0x0051), __byte_perm(u0, u1, 0x0051), 0x5410));
                }
              }
            }
            put_rows(buf, lane, w, reinterpret_cast<uint8_t*>(a.h) + (static_cast<size_t>(row0) * N + ch0) * 2,
                     static_cast<size_t>(N) * 2, rows, 2 * cols);
          } else {
            const float sx = lane < rows ? a.sx[row0 + lane] : 0.f;
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              if (c >= cols) break;
              float v[32];
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                float g[16], u[16];
                columns16(taddr + 64 * half + c + i, g);
                columns16(taddr + 128 + 64 * half + c + i, u);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const int ch = min(ch0 + c + i + j, N - 1);
                  v[i + j] = silu_mul(g[j] * (sx * __ldg(a.sw + ch)), u[j] * (sx * __ldg(a.sw1 + ch)));
                  if (c + i + j < cols) most = max_abs(most, v[i + j], 0.f);
                }
              }
              put_f32(buf, lane, v, a.hf, static_cast<size_t>(row0) * N + ch0 + c, N, rows, min(32, cols - c), true, false, true);
            }
            if (lane < rows) atomicMax(a.amax + row0 + lane, __float_as_uint(most));
          }
        }
      } else if (KIND == W_DGATED) {
        const int ch0 = tile.n * 256 + 128 * half;
        const int cols = min(128, N - ch0);
        if (rows > 0 && cols > 0) {
          const uint32_t* keep = a.saved + (static_cast<size_t>(row0 >> 5) * (N >> 1) + (ch0 >> 1)) * 96 + lane;
          uint32_t k[2][24];
          auto load = [&](int c, uint32_t (&r)[24]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const bool is = c + 2 * j < cols;
#pragma unroll
              for (int i = 0; i < 3; ++i) r[3 * j + i] = is ? __ldcs(keep + (c / 2 + j) * 96 + 32 * i) : 0u;
            }
          };
          load(0, k[0]);
          uint4 w[8];  // 32 channels: the gate's gradients, then the ups'
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            uint32_t(&r)[24] = k[(c / 16) & 1];
            if (c + 16 < 128) load(c + 16, k[(c / 16 + 1) & 1]);
            float dh[16];
            columns16(taddr + 128 * half + c, dh);
            uint32_t dg[8], du[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float o[2][2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                // (the lowest byte repeats the one above it: less than the bits that were not kept)
                const float g = __uint_as_float(__byte_perm(r[3 * j], r[3 * j + 2], i ? 0x3255 : 0x1044));
                const float u = __uint_as_float(__byte_perm(r[3 * j + 1], r[3 * j + 2], i ? 0x3277 : 0x1066));
                const float p = sigmoid(g), d = dh[2 * j + i];
                o[0][i] = d * u * (p * fmaf(g, 1.f - p, 1.f));
                o[1][i] = d * (g * p);
              }
              dg[j] = pack_bf16x2(o[0][0], o[0][1]);
              du[j] = pack_bf16x2(o[1][0], o[1][1]);
            }
            const int at = (c >> 3) & 2;
            w[at] = make_uint4(dg[0], dg[1], dg[2], dg[3]);
            w[at + 1] = make_uint4(dg[4], dg[5], dg[6], dg[7]);
            w[at + 4] = make_uint4(du[0], du[1], du[2], du[3]);
            w[at + 5] = make_uint4(du[4], du[5], du[6], du[7]);
            if ((c & 16) && c - 16 < cols) {
              const int c0 = c - 16, left = min(32, cols - c0);
#pragma unroll
              for (int i = 0; i < 8; ++i) buf[lane][i ^ (lane & 7)] = w[i];
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int row = 4 * i + (lane >> 3), piece = lane & 7;
                uint16_t* o = (piece < 4 ? a.h : a.h2) + static_cast<size_t>(row0 + row) * N + ch0 + c0 + 8 * (piece & 3);
                if (row < rows && 8 * (piece & 3) < left) *reinterpret_cast<uint4*>(o) = buf[row][piece ^ (row & 7)];
              }
              __syncwarp();
            }
          }
        }
      } else {
        const int col0 = tile.n * 256 + 128 * half;
        const int cols = min(128, N - col0);
        const long long ldy = a.ldy[tile.p];
        void* y = a.y[tile.p];
        const int size = a.out_f32 ? 4 : 2;
        const bool even = KIND != W_I8 || (ldy * size % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0);
        if (rows > 0 && cols > 0) {
          float sx = 0.f;
          if (KIND == W_I8 && lane < rows) sx = a.sx[row0 + lane];
          const bool direct = !a.out_f32 && !a.accumulate && even && (KIND != W_I8 || N % 8 == 0);
#pragma unroll
          for (int c = 0; c < 128; c += 64) {
            if (c >= cols) break;
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
              float v[32];
              columns16(taddr + 128 * half + c + i, v);
              columns16(taddr + 128 * half + c + i + 16, v + 16);
              if (KIND == W_I8) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= sx * __ldg(a.sw + min(col0 + c + i + j, N - 1));
              }
              if (direct) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[i / 8 + j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                            pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
              } else if (c + i < cols) {
                put_f32(buf, lane, v, y, static_cast<size_t>(row0) * ldy + col0 + c + i, ldy, rows, min(32, cols - c - i), a.out_f32,
                        a.accumulate, even);
              }
            }
            if (direct)
              put_rows(buf, lane, w, static_cast<uint8_t*>(y) + (static_cast<size_t>(row0) * ldy + col0 + c) * 2, ldy * 2, rows,
                       2 * min(64, cols - c));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_first(b ? tempty1 : tempty0);
      b ^= 1u;
      tphase ^= b ^ 1u;
    }
  }

  tc_fence_before();
  cluster_sync();  // nothing of either CTA is still used by the other
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

template <WKind KIND>
cudaError_t launch(const WArgs& a, cudaStream_t st) {
  const size_t smem = STAGES * STAGE + OUT_BYTES + 1024;
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(&k_wide16<KIND>), smem);
  if (e != cudaSuccess) return e;
  long long tiles = 0;
  for (int p = 0; p < (KIND == W_DW ? a.problems : 1); ++p)
    tiles += static_cast<long long>(qceil(a.m[p], 2 * BM)) * qceil(a.n[p], Kind<KIND>::cols);
  const int most = a.num_sms & ~1;
  const int grid = 2 * tiles < most ? static_cast<int>(2 * tiles) : most;
  return launch_q(k_wide16<KIND>, dim3(grid), THREADS, smem, st, a);
}

}  // namespace

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

}  // namespace pop
