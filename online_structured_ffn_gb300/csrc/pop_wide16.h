// Internal interface of the wide products of 16-bit operands (pop_wide16.cu): the gated MLP on matrices that the
// caller holds, forward and backward (pop_gated.h), and the products of 8-bit integers, which are exact in fp16
// (pop_int8.h).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pop_qinternal.h"

namespace pop {

// What a product computes. "k-major": an operand's rows have k contiguous; "mn-major": its k-th row has the M or N
// values contiguous, as a matrix that is multiplied by its other side has.
enum WKind {
  W_GATED,     // h = SiLU(A B0^T) (.) A B1^T; A, B0, B1 k-major
  W_PLAIN,     // y = A B^T; k-major
  W_DGATED,    // dh = A B (B mn-major), from it and the kept gate and up values their gradients
  W_DX,        // y = A0 B0 + A1 B1; A k-major, B mn-major
  W_DW,        // y = A^T B, up to three of them; mn-major
  W_I8,        // y = scales (.) A B^T, fp16
  W_I8_GATED,  // fp32 h from two such products, and the largest |h| of each row
};

struct WArgs {
  CUtensorMap map[6];  // A and B of each product (W_GATED: A, B0, B1; W_I8*: A), but for the A of launch_rows16
  int problems;
  int m[3], n[3];      // rows and columns of the outputs (gated: n channels)
  int kb;              // k-blocks of 64 (W_DX: of either product)
  // outputs
  void* y[3];
  long long ldy[3];
  int out_f32, accumulate;
  uint16_t* h;         // W_GATED: [m][n] bf16; W_DGATED: the gate's gradient
  uint16_t* h2;        // W_DGATED: the up values' gradient
  uint32_t* saved;     // W_GATED: what is kept of gate and up, or NULL; W_DGATED: the same
  const uint8_t* w8[2];        // W_I8*: images of the matrix (gated: of gate and up), instead of B's maps
  const float *sx, *sw, *sw1;  // W_I8*: scales of the rows, and of the columns (gated: of gate and up)
  float* hf;           // W_I8_GATED: [m][n]
  unsigned* amax;      // W_I8_GATED: bits of the largest |h| of each row (atomicMax; thin: of each tile's channels, [tile][THIN16_MOST])
  unsigned* err;
  QWait wait;
  int num_sms;
  // launch_rows16: A's rows, of k values; of few rows also, W_I8*, rows that are quantised or widened on the way:
  // `convert` 1: bf16, 2: float32 with `tiles_max` largest values of each row's parts in row_max, 3: integers with scales sx
  const void *rows, *rows2;  // (W_DX: of both products)
  long long ld_rows;
  int k;
  int convert;
  const unsigned* row_max;  // [tiles_max][THIN16_MOST]
  int tiles_max;
  int width;           // columns of a tile, as wide16_width gives them (gated: gate and up values, of half as many channels)
  int b_early;         // 1: what the kernel before this one writes is not among the B operands
  int tiles;           // set by launch_wide16
};

cudaError_t launch_wide16(WKind kind, const WArgs& a, cudaStream_t st);

// Columns of a tile. A k-major B's box has half as many rows. m, n: rows and columns of the outputs (gated: channels).
int wide16_width(WKind kind, int m, int n, int num_sms);

// All but W_DW: few rows by pop_thin16.cu, more by the wide products. (us of a whole MLP thin against wide, 4096 x 11008: bf16 65
// rows 56/66, 128 61/67; 8-bit 57/86, 70/88; 1000 x 2736 bf16 16/19, 19/20; 8192 x 28672 bf16 231/227, 244/230, 8-bit 185/219,
// 212/225. Forward and backward, the latter thin against wide: 4096 x 11008 8 rows 148/187, 100 181/203, 128 187/211; 2048 x 5496
// 57/74, 72/83, 76/87; 1000 x 2736 30/40, 45/53, 46/55.) One border for all sizes: of bf16 matrices as large as 8192 x 28672 the thin
// form of more than 64 rows is 2 to 6 % behind.
constexpr int THIN16_MOST = 128;
// CTAs to a tile of 128 outputs (pop_thin16.cu).
int thin16_split(bool i8, int m, int n, int kb, int num_sms);
// Whether a product takes its rows by `convert`: the k-blocks of a CTA have to fit beside its ring; and every CTA goes through all
// values of bf16 rows first, and there are as many CTAs as keep the device busy, so with many values a kernel of its own is
// faster (us with one and without: gate and up of 4 rows by 2 x 11008 x 4096, 16 K values, 0.5 more, of 2 rows 0.2 less; down
// projections of hidden rows, 44 K values 0.3 less, 88 K 1.0 more; 16 rows of integers by 4096 x 4096 1.0 less).
constexpr int THIN16_KEPT = 24;
bool thin16_converts(int convert, int m, int n, int k, int num_sms);
cudaError_t launch_thin16(WKind kind, const WArgs& a, cudaStream_t st);
cudaError_t launch_rows16(WKind kind, WArgs a, cudaStream_t st);

// The image of a matrix [n, k] of 8-bit integers: blocks of 128 rows by 64 k, [ceil(n/128)][ceil(k/64)][4][128][16], zeros outside.
constexpr int W8_BLOCK = 128 * 64;
inline size_t image8_bytes(int n, int k) { return static_cast<size_t>(qceil(n, 128)) * qceil(k, 64) * W8_BLOCK; }

// Kept gate and up values: for 32 rows and two channels three words a row, [ceil(m/32)][n/2][3][32]: the upper halves of
// both gates, of both ups, and the next eight bits of the four. 16 significant bits each: with 8 of them (bf16) the
// gradients were 1.7 times as far off as their own rounding makes them, with 16 1.4 times, with all 24 no less.
inline size_t saved_words(int m, int n) { return static_cast<size_t>(qceil(m, 32)) * (n / 2) * 96; }

// Tensor map of 16-bit values: `inner` contiguous ones, `outer` rows `row_bytes` apart, 128-byte swizzle, zeros outside.
bool encode_map16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes, uint32_t box_in,
                  uint32_t box_out);

enum : unsigned {
  WERR_TIMEOUT = 1u << 1,  // as QERR_TIMEOUT
};

}  // namespace pop
