/*
 * pop_quant.h — C-ABI of 8-bit operators: rows and matrices in e4m3 with a float32 scale for each block
 * of 128, their matrix product, and an MoE layer of gated-MLP experts in that format.
 *
 * The format. Rows (activations): q [M, K] e4m3 and s [M, ceil(K/128)] float32; element (m, k) stands for
 * s[m, k/128] * q[m, k]. Matrices (weights): q [N, K] e4m3 and s [ceil(N/128), ceil(K/128)] float32;
 * element (n, k) stands for s[n/128, k/128] * q[n, k]. The last block of a row or column may be short.
 *
 * Quantising a block (of a row: 128 values; of a matrix: 128 x 128): a = max(max |x|, 2^-64),
 *   s = a / 448,  q = e4m3(512 * ((0.875 * x) / a)),
 * round to nearest, ties to even, each operation in fp32. (448 = 0.875 * 512 is e4m3's largest value; for
 * bf16 x the product 0.875 x is exact, so a quotient halfway between two e4m3 values is still halfway
 * there when it is rounded.) A block that holds an infinity or a NaN stands for values that are not
 * finite (its outputs are NaN); the other rows are not touched by it.
 *
 * Products: y[m, n] = sum over blocks b of s_x[m, b] * s_w[n/128, b] * (sum over k in b of
 * q_x[m, k] * q_w[n, k]), on the tensor cores, accumulated in fp32, rounded once to y's type. The order
 * of the additions depends on the sizes (and, for the experts, on the routing) alone: the same call
 * gives the same bits.
 *
 * Conventions are those of pop_ffn.h (device pointers 16-byte aligned unless stated; stream-ordered
 * calls; status returns; device failures from the _check calls; a handle's calls must not overlap).
 * Everything a call is given lies on the current device. A handle belongs to the device that was current when
 * it was made, and its calls are refused (INVALID_ARG) while another one is.
 * Rows of x and y may lie farther apart than their length (ldx, ldy, in elements); the rows' starts
 * must be 16-byte aligned (8-byte for e4m3 rows), so the strides are multiples of 8 (bf16, e4m3) or 4
 * (float32) elements. Zero rows are allowed and do nothing.
 */
#ifndef POP_QUANT_H_
#define POP_QUANT_H_

#include "pop_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define POP_QUANT_BLOCK 128
#define POP_QUANT_MAX_DIM 65536       /* largest N and K of a matrix; K a multiple of 8, N any */
#define POP_QMOE_MAX_EXPERTS 256
#define POP_QMOE_MAX_TOP_K 16

/* Message of this thread's last failed call of this header. Never NULL. */
const char* pop_quant_last_error(void);

/* Quantises M rows of K values. x: device bf16 (x_f32 = 0) or float32 (1), rows ldx elements apart;
 * q: device e4m3, rows ldq bytes apart; s: device float32 [M, ceil(K/128)]. K: a multiple of 8, 8 to
 * 2^28 - 4096. */
pop_status pop_quantize_rows(const void* x, int x_f32, long long ldx, int M, int K, void* q, long long ldq,
                             float* s, void* stream);

/* ---- a matrix and its products */

typedef struct pop_qlinear* pop_qlinear_t;

typedef struct {
  int N, K;         /* y has N values a row, x has K; K a multiple of 8 */
  int max_tokens;   /* rows a call's workspace is made for; longer calls run in chunks of this many */
  int out_f32;      /* type of y: 1 = float32, 0 = bf16 */
} pop_qlinear_config;

/* Creates a handle on the current device that keeps its own copy of the matrix, laid out for the
 * tensor cores. W_s not NULL: W is e4m3 [N, K] with scales W_s; W_s NULL: W is bf16 [N, K] and is
 * quantised here. The caller may free W and W_s once `stream` has passed the call. Allocates the
 * workspace of later calls. On error *out is NULL. */
pop_status pop_qlinear_create(const pop_qlinear_config* cfg, const void* W, const float* W_s, void* stream,
                              pop_qlinear_t* out);

/* Frees the handle (synchronizes the device first). NULL is a no-op. */
void pop_qlinear_destroy(pop_qlinear_t h);

/* y = x W^T for M >= 0 rows of x (device bf16), which are quantised on the way. y: device [M, N], type per
 * out_f32; any alignment of its elements' size. No allocation, no host synchronization. */
pop_status pop_qlinear_forward(pop_qlinear_t h, const void* x, long long ldx, int M, void* y, long long ldy,
                               void* stream);

/* The same for rows that are in e4m3 already: xq [M, K] (rows ldq bytes apart), xs [M, ceil(K/128)]
 * (rows lds elements apart). */
pop_status pop_qlinear_forward_quantized(pop_qlinear_t h, const void* xq, long long ldq, const float* xs,
                                         long long lds, int M, void* y, long long ldy, void* stream);

/* Limit, in nanoseconds (>= 1), for every device-side wait of this handle's products from the next call on
 * (default 2 s; a captured graph keeps its own). A wait that runs out is recorded (POP_ERR_TIMEOUT from the
 * check below) and the kernel returns. The outputs of that call and of the calls after it are not valid until
 * the check has reported it; then the handle is as new. */
pop_status pop_qlinear_set_wait_limit(pop_qlinear_t h, uint64_t ns);

/* Synchronizes the device and returns the first recorded device-side failure, or POP_OK; clears it, with
 * what a wait that ran out has left in the handle. */
pop_status pop_qlinear_check(pop_qlinear_t h);

/* ---- gated-MLP experts: y_t = sum over j of w[t, j] * W2_e (quantised(SiLU(Wg_e x_t) (.) W1_e x_t)),
 * e = experts[t, j], x_t quantised, added in ascending j in fp32 */

typedef struct pop_qmoe* pop_qmoe_t;

typedef struct {
  int n_experts;   /* 1..POP_QMOE_MAX_EXPERTS (1: a dense gated MLP) */
  int top_k;       /* slots a token has, 1..POP_QMOE_MAX_TOP_K */
  int D, D_FF;     /* multiples of 8, up to POP_QUANT_MAX_DIM */
  int max_tokens;  /* tokens a call's workspace is made for; longer calls run in chunks of this many */
  int out_f32;     /* type of y: 1 = float32, 0 = bf16 */
} pop_qmoe_config;

/* Creates the layer. Wg, W1, W2: host arrays of n_experts device pointers, [D_FF, D], [D_FF, D] and
 * [D, D_FF]: e4m3 with scales Sg, S1, S2 (host arrays of device pointers), or bf16 where Sg, S1 and S2
 * are NULL. Copies the weights as pop_qlinear_create does. */
pop_status pop_qmoe_create(const pop_qmoe_config* cfg, const void* const* Wg, const void* const* W1,
                           const void* const* W2, const float* const* Sg, const float* const* S1,
                           const float* const* S2, void* stream, pop_qmoe_t* out);

void pop_qmoe_destroy(pop_qmoe_t m);

/* T >= 0 tokens x (device bf16 [T, D]); experts: device int32 [T, top_k] and weights: device float32
 * [T, top_k], as pop_route gives them. A slot of expert -1 adds nothing; any other value outside
 * [0, n_experts) adds nothing and is reported by pop_qmoe_check. One expert may stand in several of a
 * token's slots. y: device [T, D]. No allocation, no host synchronization. */
pop_status pop_qmoe_forward(pop_qmoe_t m, const void* x, long long ldx, const int* experts, const float* weights,
                            int T, void* y, long long ldy, void* stream);

/* As pop_qlinear_set_wait_limit. */
pop_status pop_qmoe_set_wait_limit(pop_qmoe_t m, uint64_t ns);

/* As pop_qlinear_check. */
pop_status pop_qmoe_check(pop_qmoe_t m);

#ifdef __cplusplus
}
#endif

#endif /* POP_QUANT_H_ */
