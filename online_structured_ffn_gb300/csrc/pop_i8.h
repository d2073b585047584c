// Internal interface of the 8-bit integer operators (include/pop_int8.h): rows and matrices (pop_i8rows.cu). Their products are
// W_I8 and W_I8_GATED of pop_wide16.h.
#pragma once
#include "pop_wide16.h"

namespace pop {

struct I8RowsArgs {
  const void* x;         // [M][ldx]
  long long ldx;
  int f32;               // 1: float32, 0: bf16
  int M, K;
  const unsigned* amax;  // bits of the rows' largest |x|, where they are known, or NULL: of `parts` parts of a row each,
  int parts;             // [parts][THIN16_MOST], or of whole rows (1)
  // outputs
  int8_t* q;             // [M][ldq], or
  uint16_t* half;        // [M][K] the same integers in fp16
  long long ldq;
  float* s;              // [M]
  unsigned* clear;       // [M] set to 0, or NULL
};
cudaError_t launch_i8_rows(const I8RowsArgs& a, cudaStream_t st);

// Integers as fp16 rows, and a copy of their scales.
cudaError_t launch_i8_half(const int8_t* q, long long ldq, const float* s, int M, int K, uint16_t* half, float* sx, cudaStream_t st);

// A matrix [N, K] of integers into its image (pop_wide16.h).
cudaError_t launch_i8_pack(const int8_t* W, int N, int K, uint8_t* image, cudaStream_t st);

}  // namespace pop
