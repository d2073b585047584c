// C ABI of the trainable gated MLP (include/pop_gated.h): argument checks, the handle, the sequences of products.
#include "pop_gated.h"

#include <new>

#include "pop_host.h"
#include "pop_wide16.h"

using namespace pop;

namespace {

thread_local std::string g_msg;

pop_status fail(pop_status s, const char* call, const char* why) noexcept { return report(g_msg, s, call, why); }
pop_status bad(const char* call, const char* why) noexcept { return report(g_msg, POP_ERR_INVALID_ARG, call, why); }
pop_status cuda(cudaError_t e, const char* call) noexcept { return report_cuda(g_msg, e, call); }

}  // namespace

struct pop_gated {  // (the pointers are of `device`)
  pop_gated_config cfg;
  uint16_t *a = nullptr, *b = nullptr;  // [max_tokens][D_FF]: h where it is not kept; gradients of gate and up
  unsigned* err = nullptr;
  QWait wait;
  int device = 0;
  int num_sms = 1;
};

namespace {

void free_gated(pop_gated* h) {
  cudaFree(h->a);
  cudaFree(h->b);
  cudaFree(h->err);
}

bool in_range(int dim) { return dim >= 8 && dim % 8 == 0 && dim <= POP_GATED_MAX_DIM; }

// Maps of a row-major matrix [outer][inner] as an operand: boxes of 64 k by `rows` where k is inner, of 64 values by 64 k where it
// is outer.
bool map_k(CUtensorMap* m, const void* p, int outer, int inner, long long ld, int rows = 128) {
  return encode_map16(m, p, inner, outer, static_cast<uint64_t>(ld) * 2, 64, rows);
}
bool map_mn(CUtensorMap* m, const void* p, int outer, int inner, long long ld) {
  return encode_map16(m, p, inner, outer, static_cast<uint64_t>(ld) * 2, 64, 64);
}

WArgs base(const pop_gated* h) {
  WArgs a{};
  a.problems = 1;
  a.err = h->err;
  a.wait = h->wait;
  a.num_sms = h->num_sms;
  return a;
}

const char* rows_wrong(const void* p, long long ld, int width, int size) {
  if (!p) return "NULL x, y or dy";
  if (off(p, 16) || ld < width || ld % (16 / size)) return "rows must start on 16-byte boundaries and be at least as far apart as they are long";
  return nullptr;
}

const uint16_t* saved_h(const void* saved, int M, int N) {
  return reinterpret_cast<const uint16_t*>(static_cast<const uint32_t*>(saved) + saved_words(M, N));
}

}  // namespace

extern "C" {

const char* pop_gated_last_error(void) { return g_msg.c_str(); }

pop_status pop_gated_create(const pop_gated_config* cfg, pop_gated_t* out) {
  const char* call = "pop_gated_create";
  if (!out) return bad(call, "out is NULL");
  *out = nullptr;
  if (!cfg) return bad(call, "cfg is NULL");
  if (!in_range(cfg->D) || !in_range(cfg->D_FF)) return bad(call, "D and D_FF must be multiples of 8 up to POP_GATED_MAX_DIM");
  if (cfg->max_tokens < 1 || cfg->max_tokens > POP_GATED_MAX_TOKENS) return bad(call, "max_tokens outside [1, 2^20]");
  if ((cfg->out_f32 | cfg->grad_f32) & ~1) return bad(call, "out_f32 and grad_f32 must be 0 or 1");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return fail(dev, call, "needs an sm_103 device");
  pop_gated* h = new (std::nothrow) pop_gated();
  if (!h) return fail(POP_ERR_OOM, call, "out of host memory");
  h->cfg = *cfg;
  h->device = current_device();
  h->num_sms = sm_count();
  const size_t n = static_cast<size_t>(cfg->max_tokens) * cfg->D_FF;
  cudaError_t e = dalloc(&h->a, n);
  if (e == cudaSuccess) e = dalloc(&h->b, n);
  if (e == cudaSuccess) e = dalloc(&h->err, 1);
  if (e == cudaSuccess) e = cudaMemset(h->err, 0, sizeof(unsigned));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();  // calls may come on streams that do not wait for this one
  if (e != cudaSuccess) {
    free_gated(h);
    delete h;
    return cuda(e, call);
  }
  *out = h;
  return POP_OK;
}

void pop_gated_destroy(pop_gated_t h) {
  if (!h) return;
  const OnDevice on(h->device);
  cudaDeviceSynchronize();
  free_gated(h);
  delete h;
}

size_t pop_gated_saved_bytes(int D_FF, int M) {
  if (!in_range(D_FF) || M < 0 || M > POP_GATED_MAX_TOKENS) return 0;
  return saved_words(M, D_FF) * 4 + static_cast<size_t>(M) * D_FF * 2;
}

static pop_status check_call(pop_gated_t h, const void* x, long long ldx, int M, const void* Wg, const void* W1, const void* W2,
                             const void* saved, const char* call) {
  if (!h) return bad(call, "NULL handle");
  if (M < 0 || M > h->cfg.max_tokens) return bad(call, "M outside [0, max_tokens]");
  if (M == 0) return POP_OK;
  if (!Wg || !W1 || !W2) return bad(call, "NULL matrix");
  if (off(Wg, 16) || off(W1, 16) || off(W2, 16) || off(saved, 16)) return bad(call, "matrices and saved must be 16-byte aligned");
  if (const char* why = rows_wrong(x, ldx, h->cfg.D, 2)) return bad(call, why);
  if (current_device() != h->device) return bad(call, "the handle was made on another device than the current one");
  return POP_OK;
}

pop_status pop_gated_forward(pop_gated_t h, const void* x, long long ldx, int M, const void* Wg, const void* W1, const void* W2,
                             void* y, long long ldy, void* saved, void* stream) {
  const char* call = "pop_gated_forward";
  const pop_status s = check_call(h, x, ldx, M, Wg, W1, W2, saved, call);
  if (s != POP_OK || M == 0) return s;
  const int D = h->cfg.D, N = h->cfg.D_FF;
  if (const char* why = rows_wrong(y, ldy, D, h->cfg.out_f32 ? 4 : 2)) return bad(call, why);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint16_t* hidden = saved ? const_cast<uint16_t*>(saved_h(saved, M, N)) : h->a;

  WArgs up = base(h);
  up.m[0] = M;
  up.n[0] = N;
  up.kb = qceil(D, 64);
  up.h = hidden;
  up.saved = static_cast<uint32_t*>(saved);
  up.rows = x;
  up.ld_rows = ldx;
  up.k = D;
  WArgs down = base(h);
  down.m[0] = M;
  down.n[0] = D;
  down.kb = qceil(N, 64);
  down.y[0] = y;
  down.ldy[0] = ldy;
  down.out_f32 = h->cfg.out_f32;
  down.b_early = 1;
  down.rows = hidden;
  down.ld_rows = N;
  down.k = N;
  if (M > THIN16_MOST) {
    up.width = wide16_width(W_GATED, M, N, h->num_sms);
    down.width = wide16_width(W_PLAIN, M, D, h->num_sms);
  }
  const int up_rows = up.width ? up.width / 2 : 128, down_rows = down.width ? down.width / 2 : 128;
  if (!map_k(&up.map[1], Wg, N, D, D, up_rows) || !map_k(&up.map[2], W1, N, D, D, up_rows) || !map_k(&down.map[1], W2, D, N, N, down_rows))
    return fail(POP_ERR_CUDA, call, "a tensor map could not be made");
  cudaError_t e = launch_rows16(W_GATED, up, st);
  if (e == cudaSuccess) e = launch_rows16(W_PLAIN, down, st);
  return cuda(e, call);
}

pop_status pop_gated_backward(pop_gated_t h, const void* x, long long ldx, int M, const void* Wg, const void* W1, const void* W2,
                              const void* saved, const void* dy, long long lddy, void* dx, long long lddx, void* dWg, void* dW1,
                              void* dW2, int accumulate, void* stream) {
  const char* call = "pop_gated_backward";
  const pop_status s = check_call(h, x, ldx, M, Wg, W1, W2, saved, call);
  if (s != POP_OK) return s;
  if (accumulate != 0 && accumulate != 1) return bad(call, "accumulate must be 0 or 1");
  if (off(dWg, 16) || off(dW1, 16) || off(dW2, 16)) return bad(call, "gradients of matrices must be 16-byte aligned");
  const int D = h->cfg.D, N = h->cfg.D_FF;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (current_device() != h->device) return bad(call, "the handle was made on another device than the current one");
    cudaError_t e = cudaSuccess;
    for (void* p : {dWg, dW1, dW2})
      if (p && !accumulate && e == cudaSuccess) e = cudaMemsetAsync(p, 0, static_cast<size_t>(D) * N * (h->cfg.grad_f32 ? 4 : 2), st);
    return cuda(e, call);
  }
  if (!saved) return bad(call, "NULL saved");
  if (const char* why = rows_wrong(dy, lddy, D, 2)) return bad(call, why);
  if (dx)
    if (const char* why = rows_wrong(dx, lddx, D, h->cfg.out_f32 ? 4 : 2)) return bad(call, why);
  const uint16_t* hidden = saved_h(saved, M, N);
  cudaError_t e = cudaSuccess;
  bool maps = true;
  if (dx || dWg || dW1) {
    WArgs a = base(h);
    a.m[0] = M;
    a.n[0] = N;
    a.kb = qceil(D, 64);
    a.h = h->a;
    a.h2 = h->b;
    a.saved = static_cast<uint32_t*>(const_cast<void*>(saved));
    a.rows = dy;
    a.ld_rows = lddy;
    a.k = D;
    maps = map_mn(&a.map[1], W2, D, N, N);
    if (maps) e = launch_rows16(W_DGATED, a, st);
  }
  if (maps && e == cudaSuccess && (dWg || dW1 || dW2)) {
    WArgs a = base(h);
    a.problems = 0;
    a.kb = qceil(M, 64);
    a.out_f32 = h->cfg.grad_f32;
    a.accumulate = accumulate;
    a.width = wide16_width(W_DW, N, D, h->num_sms);
    // The kernel in front is then the one above, which writes neither of the B operands, x and h, and lets this one start only after
    // its own wait. With dW2 alone it is one of before this call, which may write them.
    a.b_early = dx || dWg || dW1 ? 1 : 0;
    const auto add = [&](void* out, const void* left, int rows, long long ldl, const void* right, int cols, long long ldr) {
      if (!out) return;
      const int p = a.problems++;
      a.m[p] = rows;
      a.n[p] = cols;
      a.y[p] = out;
      a.ldy[p] = cols;
      maps = maps && map_mn(&a.map[2 * p], left, M, rows, ldl) && map_mn(&a.map[2 * p + 1], right, M, cols, ldr);
    };
    add(dWg, h->a, N, N, x, D, ldx);
    add(dW1, h->b, N, N, x, D, ldx);
    add(dW2, dy, D, lddy, hidden, N, N);
    if (maps) e = launch_wide16(W_DW, a, st);
  }
  if (maps && e == cudaSuccess && dx) {
    WArgs a = base(h);
    a.m[0] = M;
    a.n[0] = D;
    a.kb = qceil(N, 64);
    a.y[0] = dx;
    a.ldy[0] = lddx;
    a.out_f32 = h->cfg.out_f32;
    a.b_early = 1;
    a.rows = h->a;
    a.rows2 = h->b;
    a.ld_rows = N;
    a.k = N;
    maps = map_mn(&a.map[1], Wg, N, D, D) && map_mn(&a.map[3], W1, N, D, D);
    if (maps) e = launch_rows16(W_DX, a, st);
  }
  if (!maps) return fail(POP_ERR_CUDA, call, "a tensor map could not be made");
  return cuda(e, call);
}

pop_status pop_gated_set_wait_limit(pop_gated_t h, uint64_t ns) {
  if (!h || ns == 0) return bad("pop_gated_set_wait_limit", "NULL handle or zero limit");
  h->wait = QWait(ns);
  return POP_OK;
}

pop_status pop_gated_check(pop_gated_t h) {
  const char* call = "pop_gated_check";
  if (!h) return bad(call, "NULL handle");
  if (current_device() != h->device) return bad(call, "the handle was made on another device than the current one");
  cudaError_t e = cudaDeviceSynchronize();
  unsigned w = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&w, h->err, sizeof(w), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && w) e = cudaMemset(h->err, 0, sizeof(w));
  if (e == cudaSuccess && w) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda(e, call);
  return w ? fail(POP_ERR_TIMEOUT, call, "a wait of a product ran out") : POP_OK;
}

}  // extern "C"
