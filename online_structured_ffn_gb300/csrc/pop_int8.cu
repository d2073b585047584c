// C ABI of the 8-bit integer operators (include/pop_int8.h): argument checks, handles, workspaces, call sequences.
#include "pop_int8.h"

#include <initializer_list>
#include <new>

#include "pop_host.h"
#include "pop_i8.h"

using namespace pop;

namespace {

thread_local std::string g_msg;

pop_status fail(pop_status s, const char* call, const char* why) noexcept { return report(g_msg, s, call, why); }
pop_status bad(const char* call, const char* why) noexcept { return report(g_msg, POP_ERR_INVALID_ARG, call, why); }
pop_status cuda(cudaError_t e, const char* call) noexcept { return report_cuda(g_msg, e, call); }

constexpr int MAX_ROWS = 1 << 27;
constexpr const char* OTHER_DEVICE = "the handle was made on another device than the current one";

bool in_range(int dim) { return dim >= 8 && dim % 8 == 0 && dim <= POP_INT8_MAX_DIM; }

// A matrix [N, K] as the products take it.
struct Matrix {
  uint8_t* image = nullptr;
  float* s = nullptr;
  int N = 0, K = 0;

  cudaError_t make(const void* W, const float* W_s, int n, int k, cudaStream_t st) {
    N = n;
    K = k;
    int8_t* q = nullptr;  // of a bf16 matrix
    cudaError_t e = dalloc(&image, image8_bytes(n, k));
    if (e == cudaSuccess) e = dalloc(&s, n);
    if (W_s) {
      if (e == cudaSuccess) e = cudaMemcpyAsync(s, W_s, n * sizeof(float), cudaMemcpyDeviceToDevice, st);
    } else {
      if (e == cudaSuccess) e = dalloc(&q, static_cast<size_t>(n) * k);
      I8RowsArgs a{};
      a.x = W;
      a.ldx = k;
      a.M = n;
      a.K = k;
      a.q = q;
      a.ldq = k;
      a.s = s;
      if (e == cudaSuccess) e = launch_i8_rows(a, st);
    }
    if (e == cudaSuccess) e = launch_i8_pack(W_s ? static_cast<const int8_t*>(W) : q, n, k, image, st);
    const cudaError_t done = cudaStreamSynchronize(st);  // later calls may come on other streams; q is in use until then
    cudaFree(q);
    return e == cudaSuccess ? done : e;
  }
  void free() {
    cudaFree(image);
    cudaFree(s);
  }
};

struct Common {  // (the pointers are of `device`)
  uint16_t* rows = nullptr;  // [max_tokens][K] integers of a call's rows, in fp16
  float* sx = nullptr;
  unsigned* err = nullptr;
  QWait wait;
  int device = 0;
  int num_sms = 1;

  cudaError_t make(int max_tokens, int K) {
    device = current_device();
    num_sms = sm_count();
    cudaError_t e = dalloc(&rows, static_cast<size_t>(max_tokens) * K);
    if (e == cudaSuccess) e = dalloc(&sx, max_tokens);
    if (e == cudaSuccess) e = dalloc(&err, 1);
    if (e == cudaSuccess) e = cudaMemset(err, 0, sizeof(unsigned));
    return e == cudaSuccess ? cudaDeviceSynchronize() : e;
  }
  void free() {
    cudaFree(rows);
    cudaFree(sx);
    cudaFree(err);
  }
  pop_status check(const char* call) {
    if (current_device() != device) return bad(call, OTHER_DEVICE);
    cudaError_t e = cudaDeviceSynchronize();
    unsigned w = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&w, err, sizeof(w), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && w) e = cudaMemset(err, 0, sizeof(w));
    if (e == cudaSuccess && w) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda(e, call);
    return w ? fail(POP_ERR_TIMEOUT, call, "a wait of a product ran out") : POP_OK;
  }
  // A product with n rows of fp16 integers, [n][w.K], and their scales in sx.
  WArgs args(const Matrix& w, const uint16_t* from, int n) const {
    WArgs a{};
    a.problems = 1;
    a.m[0] = n;
    a.n[0] = w.N;
    a.kb = qceil(w.K, 64);
    a.w8[0] = w.image;
    a.sx = sx;
    a.sw = w.s;
    a.err = err;
    a.wait = wait;
    a.num_sms = num_sms;
    a.rows = from;
    a.ld_rows = w.K;
    a.k = w.K;
    return a;
  }
  // The same with rows x of bf16, quantised on the way into the product or before it. clear: [n] set to 0 by what comes before.
  cudaError_t args_of(WArgs* a, const Matrix& w, const void* x, long long ldx, int n, unsigned* clear, cudaStream_t st) const {
    *a = args(w, rows, n);
    if (thin16_converts(1, n, w.N, w.K, num_sms)) {
      a->rows = x;
      a->ld_rows = ldx;
      a->convert = 1;
      return cudaSuccess;
    }
    I8RowsArgs r{};
    r.x = x;
    r.ldx = ldx;
    r.M = n;
    r.K = w.K;
    r.half = rows;
    r.s = sx;
    r.clear = clear;
    return launch_i8_rows(r, st);
  }
};

}  // namespace

struct pop_ilinear {
  pop_ilinear_config cfg;
  Common c;
  Matrix w;
};

struct pop_iffn {
  pop_iffn_config cfg;
  Common c;
  Matrix wg, w1, w2;
  float* h = nullptr;         // [max_tokens][D_FF]
  uint16_t* hq = nullptr;     // the same, quantised, in fp16
  unsigned* amax = nullptr;   // bits of the largest |h| of each row; few rows: of each tile's channels, [tile][THIN16_MOST]
};

namespace {

void free_linear(pop_ilinear* h) {
  h->c.free();
  h->w.free();
}
void free_ffn(pop_iffn* h) {
  h->c.free();
  h->wg.free();
  h->w1.free();
  h->w2.free();
  cudaFree(h->h);
  cudaFree(h->hq);
  cudaFree(h->amax);
}

pop_status check_rows(const void* x, const void* y, int M, const char* call) {
  if (M < 0 || M > MAX_ROWS) return bad(call, "M outside [0, 2^27]");
  if (M > 0 && (!x || !y)) return bad(call, "NULL x or y");
  return POP_OK;
}

}  // namespace

extern "C" {

const char* pop_int_last_error(void) { return g_msg.c_str(); }

pop_status pop_quantize_rows_int(const void* x, int x_f32, long long ldx, int M, int K, void* q, long long ldq, float* s,
                                void* stream) {
  const char* call = "pop_quantize_rows_int";
  if (x_f32 != 0 && x_f32 != 1) return bad(call, "x_f32 must be 0 or 1");
  if (M < 0 || M > MAX_ROWS) return bad(call, "M outside [0, 2^27]");
  if (K < 8 || K % 8 || K > (1 << 30)) return bad(call, "K must be a multiple of 8 in [8, 2^30]");
  if (M == 0) return POP_OK;
  if (!x || !q || !s) return bad(call, "NULL x, q or s");
  if (off(x, 16) || off(q, 8) || off(s, 4)) return bad(call, "x must be 16-byte aligned, q 8-byte, s 4-byte");
  if (ldx < K || ldx % (x_f32 ? 4 : 8)) return bad(call, "ldx must be at least K and keep rows 16-byte aligned");
  if (ldq < K || ldq % 8) return bad(call, "ldq must be at least K and a multiple of 8");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return fail(dev, call, "needs an sm_103 device");
  I8RowsArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.f32 = x_f32;
  a.M = M;
  a.K = K;
  a.q = static_cast<int8_t*>(q);
  a.ldq = ldq;
  a.s = s;
  return cuda(launch_i8_rows(a, static_cast<cudaStream_t>(stream)), call);
}

// -------------------------------------------------------------------------------- one matrix

pop_status pop_ilinear_create(const pop_ilinear_config* cfg, const void* W, const float* W_s, void* stream, pop_ilinear_t* out) {
  const char* call = "pop_ilinear_create";
  if (!out) return bad(call, "out is NULL");
  *out = nullptr;
  if (!cfg || !W) return bad(call, "cfg or W is NULL");
  if (cfg->N < 1 || cfg->N > POP_INT8_MAX_DIM) return bad(call, "N outside [1, POP_INT8_MAX_DIM]");
  if (!in_range(cfg->K)) return bad(call, "K must be a multiple of 8 in [8, POP_INT8_MAX_DIM]");
  if (cfg->max_tokens < 1 || cfg->max_tokens > (1 << 20)) return bad(call, "max_tokens outside [1, 2^20]");
  if (cfg->out_f32 != 0 && cfg->out_f32 != 1) return bad(call, "out_f32 must be 0 or 1");
  if (off(W, 16) || off(W_s, 4)) return bad(call, "W must be 16-byte aligned, W_s 4-byte");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return fail(dev, call, "needs an sm_103 device");
  pop_ilinear* h = new (std::nothrow) pop_ilinear();
  if (!h) return fail(POP_ERR_OOM, call, "out of host memory");
  h->cfg = *cfg;
  cudaError_t e = h->c.make(cfg->max_tokens, cfg->K);
  if (e == cudaSuccess) e = h->w.make(W, W_s, cfg->N, cfg->K, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    free_linear(h);
    delete h;
    return cuda(e, call);
  }
  *out = h;
  return POP_OK;
}

void pop_ilinear_destroy(pop_ilinear_t h) {
  if (!h) return;
  const OnDevice on(h->c.device);
  cudaDeviceSynchronize();
  free_linear(h);
  delete h;
}

static pop_status linear_checked(pop_ilinear_t h, const void* x, int M, const void* y, long long ldy, const char* call) {
  if (!h) return bad(call, "NULL handle");
  const pop_status s = check_rows(x, y, M, call);
  if (s != POP_OK || M == 0) return s;
  if (ldy < h->cfg.N) return bad(call, "ldy < N");
  if (off(y, h->cfg.out_f32 ? 4 : 2)) return bad(call, "y is not aligned to its element");
  if (current_device() != h->c.device) return bad(call, OTHER_DEVICE);
  return POP_OK;
}

static uint8_t* rows_of(void* y, long long ldy, int m0, int out_f32) {
  return static_cast<uint8_t*>(y) + static_cast<size_t>(m0) * ldy * (out_f32 ? 4 : 2);
}

static cudaError_t product(pop_ilinear_t h, WArgs& a, void* y, long long ldy, int m0, cudaStream_t st) {
  a.y[0] = rows_of(y, ldy, m0, h->cfg.out_f32);
  a.ldy[0] = ldy;
  a.out_f32 = h->cfg.out_f32;
  return launch_rows16(W_I8, a, st);
}

pop_status pop_ilinear_forward(pop_ilinear_t h, const void* x, long long ldx, int M, void* y, long long ldy, void* stream) {
  const char* call = "pop_ilinear_forward";
  const pop_status s = linear_checked(h, x, M, y, ldy, call);
  if (s != POP_OK || M == 0) return s;
  if (off(x, 16) || ldx < h->cfg.K || ldx % 8) return bad(call, "x must be 16-byte aligned, ldx >= K a multiple of 8");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int m0 = 0; m0 < M; m0 += h->cfg.max_tokens) {
    const int n = M - m0 < h->cfg.max_tokens ? M - m0 : h->cfg.max_tokens;
    WArgs a;
    cudaError_t e = h->c.args_of(&a, h->w, static_cast<const uint16_t*>(x) + static_cast<size_t>(m0) * ldx, ldx, n, nullptr, st);
    if (e == cudaSuccess) e = product(h, a, y, ldy, m0, st);
    if (e != cudaSuccess) return cuda(e, call);
  }
  return POP_OK;
}

pop_status pop_ilinear_forward_quantized(pop_ilinear_t h, const void* xq, long long ldq, const float* xs, int M, void* y,
                                          long long ldy, void* stream) {
  const char* call = "pop_ilinear_forward_quantized";
  const pop_status s = linear_checked(h, xq, M, y, ldy, call);
  if (s != POP_OK || M == 0) return s;
  if (!xs || off(xs, 4)) return bad(call, "xs is NULL or misaligned");
  if (off(xq, 8) || ldq < h->cfg.K || ldq % 8) return bad(call, "xq must be 8-byte aligned, ldq >= K a multiple of 8");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int m0 = 0; m0 < M; m0 += h->cfg.max_tokens) {
    const int n = M - m0 < h->cfg.max_tokens ? M - m0 : h->cfg.max_tokens;
    const int8_t* q = static_cast<const int8_t*>(xq) + static_cast<size_t>(m0) * ldq;
    WArgs a = h->c.args(h->w, h->c.rows, n);
    cudaError_t e = cudaSuccess;
    if (thin16_converts(3, n, h->cfg.N, h->cfg.K, h->c.num_sms)) {
      a.rows = q;
      a.ld_rows = ldq;
      a.sx = xs + m0;
      a.convert = 3;
    } else {
      e = launch_i8_half(q, ldq, xs + m0, n, h->cfg.K, h->c.rows, h->c.sx, st);
    }
    if (e == cudaSuccess) e = product(h, a, y, ldy, m0, st);
    if (e != cudaSuccess) return cuda(e, call);
  }
  return POP_OK;
}

pop_status pop_ilinear_set_wait_limit(pop_ilinear_t h, uint64_t ns) {
  if (!h || ns == 0) return bad("pop_ilinear_set_wait_limit", "NULL handle or zero limit");
  h->c.wait = QWait(ns);
  return POP_OK;
}

pop_status pop_ilinear_check(pop_ilinear_t h) {
  if (!h) return bad("pop_ilinear_check", "NULL handle");
  return h->c.check("pop_ilinear_check");
}

// -------------------------------------------------------------------------------- the gated MLP

pop_status pop_iffn_create(const pop_iffn_config* cfg, const void* Wg, const void* W1, const void* W2, const float* Sg,
                            const float* S1, const float* S2, void* stream, pop_iffn_t* out) {
  const char* call = "pop_iffn_create";
  if (!out) return bad(call, "out is NULL");
  *out = nullptr;
  if (!cfg || !Wg || !W1 || !W2) return bad(call, "cfg or a matrix is NULL");
  const bool scaled = Sg || S1 || S2;
  if (scaled && (!Sg || !S1 || !S2)) return bad(call, "Sg, S1 and S2 must all be given or all be NULL");
  if (!in_range(cfg->D) || !in_range(cfg->D_FF)) return bad(call, "D and D_FF must be multiples of 8 up to POP_INT8_MAX_DIM");
  if (cfg->max_tokens < 1 || cfg->max_tokens > (1 << 20)) return bad(call, "max_tokens outside [1, 2^20]");
  if (cfg->out_f32 != 0 && cfg->out_f32 != 1) return bad(call, "out_f32 must be 0 or 1");
  if (off(Wg, 16) || off(W1, 16) || off(W2, 16) || off(Sg, 4) || off(S1, 4) || off(S2, 4))
    return bad(call, "matrices must be 16-byte aligned, scales 4-byte");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return fail(dev, call, "needs an sm_103 device");
  pop_iffn* h = new (std::nothrow) pop_iffn();
  if (!h) return fail(POP_ERR_OOM, call, "out of host memory");
  h->cfg = *cfg;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t hidden = static_cast<size_t>(cfg->max_tokens) * cfg->D_FF;
  cudaError_t e = h->c.make(cfg->max_tokens, cfg->D);
  if (e == cudaSuccess) e = dalloc(&h->h, hidden);
  if (e == cudaSuccess) e = dalloc(&h->hq, hidden);
  const size_t most = static_cast<size_t>(qceil(cfg->D_FF, 128)) * THIN16_MOST;
  if (e == cudaSuccess) e = dalloc(&h->amax, most > static_cast<size_t>(cfg->max_tokens) ? most : cfg->max_tokens);
  if (e == cudaSuccess) e = h->wg.make(Wg, Sg, cfg->D_FF, cfg->D, st);
  if (e == cudaSuccess) e = h->w1.make(W1, S1, cfg->D_FF, cfg->D, st);
  if (e == cudaSuccess) e = h->w2.make(W2, S2, cfg->D, cfg->D_FF, st);
  if (e != cudaSuccess) {
    free_ffn(h);
    delete h;
    return cuda(e, call);
  }
  *out = h;
  return POP_OK;
}

void pop_iffn_destroy(pop_iffn_t h) {
  if (!h) return;
  const OnDevice on(h->c.device);
  cudaDeviceSynchronize();
  free_ffn(h);
  delete h;
}

pop_status pop_iffn_forward(pop_iffn_t h, const void* x, long long ldx, int M, void* y, long long ldy, void* stream) {
  const char* call = "pop_iffn_forward";
  if (!h) return bad(call, "NULL handle");
  const pop_iffn_config& c = h->cfg;
  const pop_status s = check_rows(x, y, M, call);
  if (s != POP_OK || M == 0) return s;
  if (off(x, 16) || ldx < c.D || ldx % 8) return bad(call, "x must be 16-byte aligned, ldx >= D a multiple of 8");
  if (off(y, 16) || ldy < c.D || ldy % (c.out_f32 ? 4 : 8)) return bad(call, "y's rows must be 16-byte aligned, ldy >= D");
  if (current_device() != h->c.device) return bad(call, OTHER_DEVICE);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int m0 = 0; m0 < M; m0 += c.max_tokens) {
    const int n = M - m0 < c.max_tokens ? M - m0 : c.max_tokens;
    const bool thin = n <= THIN16_MOST;
    const int tiles = qceil(c.D_FF, 128);
    WArgs up;
    cudaError_t e = h->c.args_of(&up, h->wg, static_cast<const uint16_t*>(x) + static_cast<size_t>(m0) * ldx, ldx, n,
                                 thin ? nullptr : h->amax, st);
    if (e != cudaSuccess) return cuda(e, call);
    up.w8[1] = h->w1.image;
    up.sw1 = h->w1.s;
    up.hf = h->h;
    up.amax = h->amax;
    e = launch_rows16(W_I8_GATED, up, st);
    if (e != cudaSuccess) return cuda(e, call);
    WArgs down = h->c.args(h->w2, h->hq, n);
    if (thin16_converts(2, n, c.D, c.D_FF, h->c.num_sms)) {
      down.rows = h->h;
      down.convert = 2;
      down.row_max = h->amax;
      down.tiles_max = tiles;
    } else {
      I8RowsArgs hidden{};
      hidden.x = h->h;
      hidden.ldx = c.D_FF;
      hidden.f32 = 1;
      hidden.M = n;
      hidden.K = c.D_FF;
      hidden.amax = h->amax;
      hidden.parts = thin ? tiles : 1;
      hidden.half = h->hq;
      hidden.s = h->c.sx;
      e = launch_i8_rows(hidden, st);
      if (e != cudaSuccess) return cuda(e, call);
    }
    down.y[0] = rows_of(y, ldy, m0, c.out_f32);
    down.ldy[0] = ldy;
    down.out_f32 = c.out_f32;
    e = launch_rows16(W_I8, down, st);
    if (e != cudaSuccess) return cuda(e, call);
  }
  return POP_OK;
}

pop_status pop_iffn_set_wait_limit(pop_iffn_t h, uint64_t ns) {
  if (!h || ns == 0) return bad("pop_iffn_set_wait_limit", "NULL handle or zero limit");
  h->c.wait = QWait(ns);
  return POP_OK;
}

pop_status pop_iffn_check(pop_iffn_t h) {
  if (!h) return bad("pop_iffn_check", "NULL handle");
  return h->c.check("pop_iffn_check");
}

}  // extern "C"
