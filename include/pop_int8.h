/*
 * pop_int8.h — C-ABI of 8-bit integer operators: rows and matrices of integers with a float32 scale for each row
 * (token) or output channel, their product, and a gated MLP in that format.
 *
 * The format. Rows (activations): q [M, K] int8 and s [M] float32; element (m, k) stands for s[m] * q[m, k]. Matrices
 * (weights): q [N, K] int8 and s [N] float32; element (n, k) stands for s[n] * q[n, k].
 *
 * Quantising a row: a = max(max |x|, 2^-64), s = a / 127, q = rint(128 * ((127/128 * x) / a)), halves to even, each
 * operation in fp32. (For bf16 x the product 127/128 x is exact, so a quotient halfway between two integers is still
 * halfway there when it is rounded.) A row that holds an infinity or a NaN gets the scale NaN and zeros: its outputs are
 * NaN; the other rows are not touched by it. q is never -128 then, but may be where it is given.
 *
 * Products: y[m, n] = s_x[m] * s_w[n] * (sum over k of q_x[m, k] * q_w[n, k]). The integers are exact in fp16 and so are
 * their products; they are summed in fp32 on the tensor cores, exactly as long as no partial sum passes 2^24. Beyond that an
 * addition may be cut off at 2^-23 of the partial sum, so the error grows with K: at most K 2^-23 of the sum of the products'
 * magnitudes. (sm_103a has no tensor-core product of 8-bit integers: the format saves memory, and time where the matrix's bytes
 * are what a call takes; many rows take no less time than in bf16, and more than in e4m3, pop_quant.h.) y is rounded once to its
 * type. The order of the additions depends on the sizes alone: the same call gives the same bits.
 *
 * Conventions are those of pop_ffn.h (device pointers 16-byte aligned unless stated; stream-ordered calls; status returns;
 * device failures from the _check calls; a handle's calls must not overlap). Everything a call is given lies on the
 * current device. A handle belongs to the device that was current when it was made, and its calls are refused
 * (INVALID_ARG) while another one is. Rows of x and y may lie farther apart than their length (ld*, in elements); rows
 * of bf16 and float32 must start on 16-byte boundaries, of integers on 8-byte ones. Zero rows are allowed and do
 * nothing. Outputs must not overlap inputs.
 */
#ifndef POP_INT8_H_
#define POP_INT8_H_

#include "pop_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define POP_INT8_MAX_DIM 65536    /* largest N and K of a matrix; K a multiple of 8, N any */

/* Message of this thread's last failed call of this header. Never NULL. */
const char* pop_int_last_error(void);

/* Quantises M rows of K values. x: device bf16 (x_f32 = 0) or float32 (1), rows ldx elements apart; q: device int8, rows
 * ldq apart; s: device float32 [M]. K: a multiple of 8, 8 to 2^30. */
pop_status pop_quantize_rows_int(const void* x, int x_f32, long long ldx, int M, int K, void* q, long long ldq, float* s,
                                void* stream);

/* ---- a matrix and its products */

typedef struct pop_ilinear* pop_ilinear_t;

typedef struct {
  int N, K;         /* y has N values a row, x has K; K a multiple of 8 */
  int max_tokens;   /* rows a call's workspace is made for; longer calls run in chunks of this many */
  int out_f32;      /* type of y: 1 = float32, 0 = bf16 */
} pop_ilinear_config;

/* Creates a handle on the current device that keeps its own copy of the matrix, laid out for the products. W_s not NULL:
 * W is int8 [N, K] with scales W_s [N]; W_s NULL: W is bf16 [N, K] and is quantised here, a row at a time. The caller may
 * free W and W_s when the call returns (it waits for `stream`). Allocates the workspace of later calls. On error *out is
 * NULL. */
pop_status pop_ilinear_create(const pop_ilinear_config* cfg, const void* W, const float* W_s, void* stream, pop_ilinear_t* out);

/* Frees the handle (synchronizes the device first). NULL is a no-op. */
void pop_ilinear_destroy(pop_ilinear_t h);

/* y = x W^T for M >= 0 rows of x (device bf16), which are quantised on the way. y: device [M, N], type per out_f32; any
 * alignment of its elements' size. No allocation, no host synchronization; may be captured in a CUDA graph. */
pop_status pop_ilinear_forward(pop_ilinear_t h, const void* x, long long ldx, int M, void* y, long long ldy, void* stream);

/* The same for rows that are integers already: xq [M, K] (rows ldq bytes apart), xs [M]. */
pop_status pop_ilinear_forward_quantized(pop_ilinear_t h, const void* xq, long long ldq, const float* xs, int M, void* y,
                                          long long ldy, void* stream);

/* Limit, in nanoseconds (>= 1), for every device-side wait of this handle's products from the next call on (default 2 s; a
 * captured graph keeps its own). A wait that runs out is recorded (POP_ERR_TIMEOUT from the check below) and the kernel
 * returns. The outputs of that call and of the calls after it are not valid until the check has reported it. */
pop_status pop_ilinear_set_wait_limit(pop_ilinear_t h, uint64_t ns);

/* Synchronizes the device and returns the first recorded device-side failure, or POP_OK; clears it. */
pop_status pop_ilinear_check(pop_ilinear_t h);

/* ---- a gated MLP: y = W2 quantised(SiLU(Wg x') (.) (W1 x')), x' = quantised(x); the hidden rows are fp32 until they are
 * quantised */

typedef struct pop_iffn* pop_iffn_t;

typedef struct {
  int D, D_FF;      /* multiples of 8, up to POP_INT8_MAX_DIM */
  int max_tokens;   /* tokens a call's workspace is made for (6 * max_tokens * D_FF bytes and more); longer calls run in
                       chunks of this many */
  int out_f32;      /* type of y: 1 = float32, 0 = bf16 */
} pop_iffn_config;

/* Creates the layer. Wg, W1: [D_FF, D], W2: [D, D_FF]: int8 with scales Sg, S1 [D_FF] and S2 [D], or bf16 where Sg, S1 and
 * S2 are NULL. Copies the weights as pop_ilinear_create does. */
pop_status pop_iffn_create(const pop_iffn_config* cfg, const void* Wg, const void* W1, const void* W2, const float* Sg,
                            const float* S1, const float* S2, void* stream, pop_iffn_t* out);

void pop_iffn_destroy(pop_iffn_t h);

/* M >= 0 tokens x (device bf16 [M, D]) to y (device [M, D]; rows 16-byte aligned). No allocation, no host synchronization;
 * may be captured in a CUDA graph. */
pop_status pop_iffn_forward(pop_iffn_t h, const void* x, long long ldx, int M, void* y, long long ldy, void* stream);

/* As of pop_ilinear. */
pop_status pop_iffn_set_wait_limit(pop_iffn_t h, uint64_t ns);
pop_status pop_iffn_check(pop_iffn_t h);

#ifdef __cplusplus
}
#endif

#endif /* POP_INT8_H_ */
