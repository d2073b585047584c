// Internal interface of the routing and 8-bit operators (pop_route.h, pop_quant.h).
//
// Operand images. The 8-bit products take both operands as shared-memory images: a k-block (128 values
// of k) of a run of rows is `rows` x 128 bytes in the 128-byte swizzle (row r's 16-byte chunk c lies at
// chunk c ^ (r % 8)), one contiguous piece of memory that a bulk copy brings into place as it is.
//   - a matrix [N, K]: tiles of 128 rows, [ceil(N/128)][ceil(K/128)][16 KB]; rows past N and bytes past K
//     are zero. Its scales are float32, a tile's ceil(K/128) in order, tiles scale_stride apart. The gate and
//     up matrices of a gated MLP share one image, [tile][k-block][gate 16 KB | up 16 KB], and their scales
//     [tile][k-block][2].
//   - rows (tokens): runs of G rows (G = 16, 32, 64 or 128), [run][k-block][G x 128 bytes]; scales
//     [run][k-block][G]. Bytes past K are zero; what rows without a token hold is not used.
// Tokens of an expert stand together, in ascending order, and every expert's begin a run.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "pop_quant.h"

namespace pop {

// Launches a kernel. The status is this launch's own; cudaGetLastError would also give what an earlier call has left.
template <class K, class... Args>
cudaError_t launch_plain(K kernel, dim3 grid, int block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// POP_OK if the current device is a GB300 (sm_103). Looked up once per device.
pop_status device_supported();

constexpr int QB = 128;              // block of a scale, and of an operand image in k
constexpr int QTILE = QB * QB;       // bytes of a 128 x 128 image
__host__ __device__ constexpr int qceil(int a, int b) { return (a + b - 1) / b; }
// Floats from one tile's scales to the next one's: whole runs of eight k-blocks, which bulk copies bring in.
__host__ __device__ constexpr int scale_stride(int KB, int step) { return qceil(KB, 8) * 8 * step; }
// Floats that a copy of eight k-blocks' scales may reach past the last tile's.
constexpr int SCALE_PAD = 16;

// Byte of (row, k) within an image of 128-byte rows.
__host__ __device__ constexpr uint32_t image_at(uint32_t row, uint32_t k) {
  return row * 128u + ((((k >> 4) ^ row) & 7u) << 4) + (k & 15u);
}

struct QRowsArgs {       // rows to quantise, or in e4m3 already
  const void* x;
  long long ldx;         // elements between rows
  int kind;              // 0 bf16, 1 float32, 2 e4m3 with scales xs
  const float* xs;
  long long lds;
  int M, K;
};
struct QRowsOut {
  uint8_t* q;            // plain: [M][ldq]; image: runs of G rows
  float* s;              // plain: [M][KB]; image: [run][KB][G]
  long long ldq;
  int G;                 // 0: plain
  // image: rows of token t (NULL: row t itself): row_of[t * k + j] for j < k, < 0 for none
  const int* row_of;
  int k;
  // few pairs: the places are found on the way, from the experts of all pairs, and written to places
  const int* experts;
  int E;
  int* places;
  unsigned* err;
};
cudaError_t launch_quantize_rows(const QRowsArgs& in, const QRowsOut& out, cudaStream_t st);

// One matrix [N, K] (e4m3 with scales Ws, or bf16 with Ws NULL) into its place in an image: tile t,
// k-block b goes to img + ((t * KB + b) * step + part) * QTILE, its scale to
// s[t * scale_stride(KB, step) + b * step + part].
cudaError_t launch_pack_matrix(const void* W, const float* Ws, int N, int K, uint8_t* img, float* s, int step,
                               int part, cudaStream_t st);

// Groups the pairs (token, slot) by expert: counts[e] and every pair's row, in ascending pair order within an expert,
// each expert beginning a run of G rows; -1 for a pair without an expert. For up to FEW_PAIRS pairs no kernel of its
// own is needed: the quantiser finds the places and the products count, every CTA for itself (calls of a graph with and
// without the kernel: one token through 8 experts 70.6 and 66.0 us, 1998 pairs over 64 experts 110.9 and 108.0, 4096
// over 8 46.8 and 50.3).
constexpr int FEW_PAIRS = 2048;
cudaError_t launch_plan(const int* experts, int pairs, int E, int G, int* counts, int* row_of, unsigned* err,
                        cudaStream_t st);

// y[t] = sum over j of weights[t, j] * o[row_of[t, j]]
cudaError_t launch_combine(const float* o, const int* row_of, const float* weights, int T, int k, int D, void* y,
                           long long ldy, int out_f32, cudaStream_t st);

// Limit of a wait: the timer is read after 64 tries, as reading it takes longer than most waits; after every one if
// the limit is shorter than some hundred tries.
struct QWait {
  uint64_t ns;
  uint32_t more;  // tries between two looks, less one: 2^n - 1
  __host__ __device__ constexpr QWait(uint64_t limit = 2000000000ull) : ns(limit), more(limit < 100000u ? 0u : 63u) {}
};

struct QGemmArgs {
  const uint8_t* act;    // rows
  const float* act_s;
  int G;
  const uint8_t* w;      // E matrices (gated: E gate/up images), w_stride bytes apart
  const float* ws;       // ws_stride floats apart
  size_t w_stride, ws_stride;
  int N, K;
  int E;                 // groups: experts, or 1
  const int* counts;     // device [E] rows of each group; or
  const int* experts;    // device [M] experts of all pairs, which are counted here; both NULL: one group of M rows
  int M;                 // rows in all, as far as the host knows: the exact number, or the number of pairs
  const QRowsArgs* rows; // thin, one group of up to 16 rows: the rows themselves (kind 0 or 2), which the kernel
                         // quantises on the way instead of taking act and act_s; or NULL
  // outputs. gated: rows in e4m3 for the next product (same G and rows); else y
  uint8_t* h;
  float* h_s;
  void* y;
  long long ldy;
  int out_f32;
  // parts of tiles that several CTAs share (qgemm_thin_parts or qgemm_wide_parts floats), and a counter per tile
  // (thin; wide: per SM), zero between calls
  float* parts;
  unsigned* done;
  unsigned* err;
  QWait wait;            // limit of the kernel's waits
  int num_sms;
};
// few rows per group (G = 16, 32 or 64): the matrix streams once (pop_qthin.cu)
cudaError_t launch_qgemm_thin(const QGemmArgs& a, bool gated, cudaStream_t st);
size_t qgemm_thin_parts(int num_sms, bool gated);
// many rows per group (G = 128): 128 x 256 tiles (pop_qwide.cu)
cudaError_t launch_qgemm_wide(const QGemmArgs& a, bool gated, cudaStream_t st);
size_t qgemm_wide_parts(int num_sms);

enum : unsigned {
  QERR_EXPERT = 1u << 0,   // an expert index outside [-1, n_experts)
  QERR_TIMEOUT = 1u << 1,  // a wait of a product ran out
};

}  // namespace pop
