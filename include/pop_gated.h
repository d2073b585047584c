/*
 * pop_gated.h — C-ABI of the gated MLP on matrices that the caller holds and trains: forward, and the
 * backward pass. (pop_ffn.h packs the weights of a layer that is only run, and prunes it.)
 *
 * For rows x (M of D values), Wg and W1 [D_FF, D] and W2 [D, D_FF], p the logistic function 1 / (1 + exp(-g)):
 *   forward    g = x Wg^T,  u = x W1^T,  h = SiLU(g) (.) u = g p (.) u,  y = h W2^T
 *   backward   for dy, the gradient of a loss in y:
 *              dh = dy W2,  dg = dh (.) u (.) p (1 + g (1 - p)),  du = dh (.) g p,
 *              dx = dg Wg + du W1,  dWg = dg^T x,  dW1 = du^T x,  dW2 = dy^T h
 *
 * x, dy and the matrices are bf16. The products run on the tensor cores and are summed in fp32; the activation
 * and its derivative are fp32. What one product hands to the next as an operand (h, dg, du) is rounded to bf16, once;
 * forward keeps g and u for backward with 16 significant bits (they are cut off there, an error below 2^-15) and h in
 * bf16. Outputs are rounded once to their type: out_f32 and grad_f32 spare that rounding, not those of h, dg and du (an
 * output is 2.4e-3 of its norm from the definition in bf16, 1.7e-3 of it by its own rounding, 1.7e-3 in float32). The order of
 * the additions depends on the sizes alone: the same call gives the same bits, and a gradient those that it has whichever
 * others are asked for. A row of x or dy that is not finite gives gradients of the matrices that are not; of y and
 * dx it touches its own row alone.
 *
 * Conventions are those of pop_ffn.h (device pointers 16-byte aligned; stream-ordered calls; status returns; device
 * failures from pop_gated_check; a handle's calls must not overlap). Everything a call is given lies on the current
 * device. A handle belongs to the device that was current when it was made, and its calls are refused
 * (INVALID_ARG) while another one is. It holds no weights: one handle serves any number of layers of its sizes.
 * Rows of x, y, dy and dx may lie farther apart than their length (ld*, in elements); their starts must be 16-byte
 * aligned. Matrices and their gradients are contiguous. Outputs must not overlap inputs or one another.
 */
#ifndef POP_GATED_H_
#define POP_GATED_H_

#include "pop_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define POP_GATED_MAX_DIM 65536       /* largest D and D_FF, multiples of 8 */
#define POP_GATED_MAX_TOKENS (1 << 20)

typedef struct pop_gated* pop_gated_t;

typedef struct {
  int D, D_FF;      /* multiples of 8, 8..POP_GATED_MAX_DIM */
  int max_tokens;   /* largest M of a call, 1..POP_GATED_MAX_TOKENS; the workspace is 4 * max_tokens * D_FF bytes */
  int out_f32;      /* type of y and dx: 1 = float32, 0 = bf16 */
  int grad_f32;     /* type of dWg, dW1 and dW2: 1 = float32, 0 = bf16 */
} pop_gated_config;

/* Creates a handle on the current device. Errors: INVALID_ARG, UNSUPPORTED (not sm_103), OOM, CUDA; then *out is
 * NULL. */
pop_status pop_gated_create(const pop_gated_config* cfg, pop_gated_t* out);

/* Frees the handle (synchronizes the device first). NULL is a no-op. */
void pop_gated_destroy(pop_gated_t h);

/* Bytes that forward keeps of M rows for backward (a buffer of the caller's). 0 if M or D_FF is out of range. */
size_t pop_gated_saved_bytes(int D_FF, int M);

/* y for 0 <= M <= max_tokens rows. saved: a device buffer of pop_gated_saved_bytes(D_FF, M), for backward, or NULL.
 * Two kernels; no allocation, no host synchronization; may be captured in a CUDA graph. */
pop_status pop_gated_forward(pop_gated_t h, const void* x, long long ldx, int M, const void* Wg, const void* W1,
                             const void* W2, void* y, long long ldy, void* saved, void* stream);

/* The gradients of the call that filled `saved`, for the same x, M and matrices. dy is bf16 whatever y's type. dx, dWg, dW1, dW2: any of them may be
 * NULL and is then not computed. accumulate 1: the matrices' gradients are added to what dWg, dW1 and dW2 hold (in fp32,
 * before the rounding to their type); 0: they are overwritten, with M = 0 by zeros. `saved` is only read: a
 * second call gives the same. */
pop_status pop_gated_backward(pop_gated_t h, const void* x, long long ldx, int M, const void* Wg, const void* W1,
                              const void* W2, const void* saved, const void* dy, long long lddy, void* dx, long long lddx,
                              void* dWg, void* dW1, void* dW2, int accumulate, void* stream);

/* Limit, in nanoseconds (>= 1), for every device-side wait of this handle's kernels from the next call on (default
 * 2 s; a captured graph keeps its own). A wait that runs out is recorded (POP_ERR_TIMEOUT from the check below) and
 * the kernel returns; the outputs of that call and of the calls after it are not valid until the check has reported
 * it. */
pop_status pop_gated_set_wait_limit(pop_gated_t h, uint64_t ns);

/* Synchronizes the device and returns the first recorded device-side failure, or POP_OK; clears it. */
pop_status pop_gated_check(pop_gated_t h);

/* Message of this thread's last failed call of this header. Never NULL. */
const char* pop_gated_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* POP_GATED_H_ */
