// C ABI of the 8-bit operators (include/pop_quant.h): argument checks, handles, workspaces, call sequences.
#include "pop_quant.h"

#include <atomic>
#include <cmath>
#include <initializer_list>
#include <mutex>
#include <new>
#include <string>

#include "pop_host.h"
#include "pop_qinternal.h"

namespace {

thread_local std::string g_quant_msg;

pop_status q_fail(pop_status s, const char* call, const char* why) noexcept { return pop::report(g_quant_msg, s, call, why); }

pop_status q_cuda(cudaError_t e, const char* call) noexcept { return pop::report_cuda(g_quant_msg, e, call); }

using pop::current_device;
using pop::dalloc;
using pop::off;
using pop::OnDevice;
using pop::sm_count;

// A handle's calls launch on the current device, with its pointers.
pop_status same_device(int device, const char* call) {
  if (current_device() == device) return POP_OK;
  return q_fail(POP_ERR_INVALID_ARG, call, "the handle was made on another device than the current one");
}

constexpr long long MAX_ROWS = 1ll << 27;
constexpr int MAX_ROW = 65535 * 32 * pop::QB;  // values that a grid's second dimension holds, of 32 blocks each

// The device error word's first failure. After a wait that ran out the tiles' counters hold what the CTAs that gave up
// left unfinished: they are cleared with it, or later calls would sum parts that are not there yet.
pop_status check_word(unsigned* err, unsigned* done, size_t counters, const char* call) {
  cudaError_t e = cudaDeviceSynchronize();
  unsigned w = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&w, err, sizeof(w), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return q_cuda(e, call);
  if (!w) return POP_OK;
  if (w & pop::QERR_TIMEOUT) e = cudaMemset(done, 0, counters * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(err, 0, sizeof(w));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();  // later calls may come on streams that do not wait for this one
  if (e != cudaSuccess) return q_cuda(e, call);
  if (w & pop::QERR_TIMEOUT) return q_fail(POP_ERR_TIMEOUT, call, "a wait of a product ran out");
  return q_fail(POP_ERR_DEVICE, call, "an expert index outside [-1, n_experts)");
}

}  // namespace

namespace pop {

pop_status device_supported() {
  static std::atomic<int> known[64];  // 0 unknown, 1 supported, 2 not
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return POP_ERR_CUDA;
  const bool tracked = dev >= 0 && dev < 64;
  int k = tracked ? known[dev].load(std::memory_order_relaxed) : 0;
  if (k == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return POP_ERR_CUDA;
    k = major == 10 && minor == 3 ? 1 : 2;
    if (tracked) known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 1 ? POP_OK : POP_ERR_UNSUPPORTED;
}

}  // namespace pop

using namespace pop;

struct pop_qlinear {  // (the pointers are of `device`)
  pop_qlinear_config cfg;
  uint8_t* w = nullptr;    // matrix image
  float* ws = nullptr;
  uint8_t* act = nullptr;  // image of a call's rows
  float* act_s = nullptr;
  float* parts = nullptr;
  unsigned* done = nullptr;
  size_t counters = 0;     // of done
  unsigned* err = nullptr;
  QWait wait;
  int device = 0;
  int num_sms = 1;
};

struct pop_qmoe {
  pop_qmoe_config cfg;
  uint8_t *wgu = nullptr, *wdn = nullptr;
  float *sgu = nullptr, *sdn = nullptr;
  int *counts = nullptr, *row_of = nullptr;
  uint8_t *act = nullptr, *h = nullptr;
  float *act_s = nullptr, *h_s = nullptr;
  float* o = nullptr;      // [rows][D] outputs of the experts
  float* parts = nullptr;
  unsigned* done = nullptr;
  size_t counters = 0;     // of done
  unsigned* err = nullptr;
  QWait wait;
  int device = 0;
  int num_sms = 1;
};

namespace {

// One product of the experts or of a matrix, for the choice between its two kernels: `groups` groups of about `rows`
// rows, NT tiles of 128 outputs (gated: of channels), KB k-blocks.
struct Shape {
  long long groups, rows;
  int NT, KB;
  bool gated;
};

// Times of the two kernels, in 0.05 us. Wide: rounds of 256 x 256 tiles over pairs of SMs, a k-block 0.35 us, or 0.5
// where a matrix tile serves one row tile only and comes from memory. Thin: tiles of 64 rows by 128 outputs over all SMs, a
// k-block 0.36 us (gated: two products, 0.8 us) and a little more, as the matrix is read again for every further
// tile of rows. Measured, rows per group, thin against wide in us: 8 experts of 2 x 14336 x 4096 64: 143/183, 80: 274/183;
// 28672 x 8192 64: 43/56, 80: 76/56; 11008 x 4096 64: 16/17, 80: 19/17; 1000 x 8000 64: 13/27, 256: 14/29; 64 experts of
// 2 x 1000 x 2048 64: 52/61, 80: 77/62, of 2048 x 1000 64: 36/44, 80: 49/45.
double wide_time(const Shape& s, int sms) {
  const long long tiles = s.groups * ((s.rows + 255) / 256) * (s.gated ? s.NT : qceil(s.NT, 2));
  return static_cast<double>((tiles + sms / 2 - 1) / (sms / 2)) * s.KB * (s.rows <= 256 ? 10 : 7);
}
double thin_time(const Shape& s, int sms) {
  return static_cast<double>(s.groups * ((s.rows + 63) / 64) * s.NT) * s.KB * (s.gated ? 20 : 10) / sms;
}

// Rows of a group above which no call is thin, so that the tiles' counters have a bound. The times above would choose thin
// beyond it only by few outputs, where it hardly matters (thin/wide in us: 1025 rows by 8 x 4096 15.9/17.6, 4096 by 8 x 4096
// 23.7/23.9, 4096 by 128 x 2048 17.1/16.0).
constexpr long long THIN_MOST = 1024;

// Rows of a run, which says which kernel a call takes: 128 (wide), else thin with tiles of as many rows as a group can
// have if a token is in it once, up to 64.
int granule(std::initializer_list<Shape> products, int tokens, int sms) {
  double wide = 0, thin = 0;
  bool few = true;
  for (const Shape& s : products) {
    wide += wide_time(s, sms);
    thin += thin_time(s, sms);
    few = few && s.rows <= THIN_MOST;
  }
  return !few || thin > wide ? 128 : tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
}

// Counters of the tiles that CTAs share. Thin: row tiles (of 16 at least; of 64 with more than 32 tokens) of all groups,
// times output tiles. Wide: one per SM.
size_t tile_counters(long long pairs, long long few_pairs, int E, size_t out_tiles, int num_sms) {
  const long long most = THIN_MOST * E < pairs ? THIN_MOST * E : pairs;
  const long long used = most < E ? most : E;
  const long long many = most / 64 + used, few = few_pairs / 16 + used;
  const size_t thin = static_cast<size_t>(many > few ? many : few) * out_tiles;
  return thin > static_cast<size_t>(num_sms) ? thin : num_sms;
}
// Floats of their parts.
size_t part_floats(bool wide, bool gated, int num_sms) {
  const size_t t = qgemm_thin_parts(num_sms, gated), w = wide ? qgemm_wide_parts(num_sms) : 0;
  return t > w ? t : w;
}

cudaError_t launch_qgemm(const QGemmArgs& g, bool gated, cudaStream_t st) {
  return g.G == 128 ? launch_qgemm_wide(g, gated, st) : launch_qgemm_thin(g, gated, st);
}

void free_linear(pop_qlinear* h) {
  cudaFree(h->w);
  cudaFree(h->ws);
  cudaFree(h->act);
  cudaFree(h->act_s);
  cudaFree(h->parts);
  cudaFree(h->done);
  cudaFree(h->err);
}

void free_qmoe(pop_qmoe* m) {
  void* p[] = {m->wgu, m->wdn, m->sgu, m->sdn, m->counts, m->row_of, m->act, m->h, m->act_s, m->h_s, m->o, m->parts, m->done, m->err};
  for (void* q : p) cudaFree(q);
}

int linear_granule(const pop_qlinear_config& c, int rows, int sms) {
  return granule({{1, rows, qceil(c.N, QB), qceil(c.K, QB), false}}, rows, sms);
}

// The experts' rows spread about their mean, by two deviations of a random routing: some pass 64 when the mean is at 50.
// (Mean rows per expert, thin against wide, both products of a call, in us: 8 experts of 4096 x 14336 48: 280/273, 52: 306/275;
// 64 of 2048 x 1000 48: 116/128, 52: 123/129, 60: 133/132; 16 of 1024 x 1024 52: 34/29.)
int qmoe_granule(const pop_qmoe_config& c, int tokens, int sms) {
  const long long pairs = static_cast<long long>(tokens) * c.top_k;
  const long long groups = pairs < c.n_experts ? pairs : c.n_experts;
  const long long mean = groups ? (pairs + groups - 1) / groups : 0;
  const long long rows = c.n_experts > 1 ? mean + static_cast<long long>(2 * std::sqrt(static_cast<double>(mean))) : pairs;
  const int NT = qceil(c.D_FF, QB), DT = qceil(c.D, QB);
  return granule({{groups, rows, NT, DT, true}, {groups, rows, DT, NT, false}}, tokens, sms);
}

pop_status linear_call(pop_qlinear* h, QRowsArgs in, size_t row_bytes, int M, void* y, long long ldy, cudaStream_t st,
                       const char* call) {
    for (int m0 = 0; m0 < M; m0 += h->cfg.max_tokens) {
    const int n = M - m0 < h->cfg.max_tokens ? M - m0 : h->cfg.max_tokens;
    const int G = linear_granule(h->cfg, n, h->num_sms);
    QRowsArgs part = in;
    part.x = static_cast<const uint8_t*>(in.x) + static_cast<size_t>(m0) * in.ldx * row_bytes;
    if (in.xs) part.xs = in.xs + static_cast<size_t>(m0) * in.lds;
    part.M = n;
    QGemmArgs g{};
    cudaError_t e = cudaSuccess;
    if (n <= 16 && G == 16) {
      g.rows = &part;  // quantised on the way into the product
    } else {
      QRowsOut o{};
      o.q = h->act;
      o.s = h->act_s;
      o.G = G;
      o.k = 1;
      e = launch_quantize_rows(part, o, st);
      if (e != cudaSuccess) return q_cuda(e, call);
    }
    g.act = h->act;
    g.act_s = h->act_s;
    g.G = G;
    g.w = h->w;
    g.ws = h->ws;
    g.N = h->cfg.N;
    g.K = h->cfg.K;
    g.E = 1;
    g.M = n;
    g.y = static_cast<uint8_t*>(y) + static_cast<size_t>(m0) * ldy * (h->cfg.out_f32 ? 4 : 2);
    g.ldy = ldy;
    g.out_f32 = h->cfg.out_f32;
    g.parts = h->parts;
    g.done = h->done;
    g.err = h->err;
    g.wait = h->wait;
    g.num_sms = h->num_sms;
    e = launch_qgemm(g, false, st);
    if (e != cudaSuccess) return q_cuda(e, call);
  }
  return POP_OK;
}

}  // namespace

extern "C" {

const char* pop_quant_last_error(void) { return g_quant_msg.c_str(); }

pop_status pop_quantize_rows(const void* x, int x_f32, long long ldx, int M, int K, void* q, long long ldq, float* s,
                             void* stream) {
  const char* call = "pop_quantize_rows";
  const auto bad = [&](const char* why) { return q_fail(POP_ERR_INVALID_ARG, call, why); };
  if (x_f32 != 0 && x_f32 != 1) return bad("x_f32 must be 0 or 1");
  if (M < 0 || M > MAX_ROWS) return bad("M outside [0, 2^27]");
  if (K < 8 || K % 8 || K > MAX_ROW) return bad("K must be a multiple of 8 in [8, 2^28 - 4096]");
  if (M == 0) return POP_OK;
  if (!x || !q || !s) return bad("NULL x, q or s");
  if (off(x, 16) || off(q, 8) || off(s, 4)) return bad("x must be 16-byte aligned, q 8-byte, s 4-byte");
  if (ldx < K || ldx % (x_f32 ? 4 : 8)) return bad("ldx must be at least K and keep rows 16-byte aligned");
  if (ldq < K || ldq % 8) return bad("ldq must be at least K and a multiple of 8");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return q_fail(dev, call, "needs an sm_103 device");
  QRowsArgs in{x, ldx, x_f32, nullptr, 0, M, K};
  QRowsOut out{};
  out.q = static_cast<uint8_t*>(q);
  out.s = s;
  out.ldq = ldq;
  return q_cuda(launch_quantize_rows(in, out, static_cast<cudaStream_t>(stream)), call);
}

// -------------------------------------------------------------------------------- one matrix

pop_status pop_qlinear_create(const pop_qlinear_config* cfg, const void* W, const float* W_s, void* stream,
                              pop_qlinear_t* out) {
  const char* call = "pop_qlinear_create";
  const auto bad = [&](const char* why) { return q_fail(POP_ERR_INVALID_ARG, call, why); };
  if (!out) return bad("out is NULL");
  *out = nullptr;
  if (!cfg || !W) return bad("cfg or W is NULL");
  if (cfg->N < 1 || cfg->N > POP_QUANT_MAX_DIM) return bad("N outside [1, POP_QUANT_MAX_DIM]");
  if (cfg->K < 8 || cfg->K % 8 || cfg->K > POP_QUANT_MAX_DIM)
    return bad("K must be a multiple of 8 in [8, POP_QUANT_MAX_DIM]");
  if (cfg->max_tokens < 1 || cfg->max_tokens > (1 << 20)) return bad("max_tokens outside [1, 2^20]");
  if (cfg->out_f32 != 0 && cfg->out_f32 != 1) return bad("out_f32 must be 0 or 1");
  if (off(W, 16) || off(W_s, 4)) return bad("W must be 16-byte aligned");
  const pop_status dev = device_supported();
  if (dev != POP_OK) return q_fail(dev, call, "needs an sm_103 device");
  pop_qlinear* h = new (std::nothrow) pop_qlinear();
  if (!h) return q_fail(POP_ERR_OOM, call, "out of host memory");
  h->cfg = *cfg;
  h->device = current_device();
  h->num_sms = sm_count();
  const size_t rows = static_cast<size_t>(qceil(cfg->max_tokens, 128)) * 128;
  const size_t NT = qceil(cfg->N, QB), KB = qceil(cfg->K, QB);
  cudaError_t e = dalloc(&h->w, NT * KB * QTILE);
  if (e == cudaSuccess) e = dalloc(&h->ws, NT * scale_stride(KB, 1) + SCALE_PAD);
  if (e == cudaSuccess) e = dalloc(&h->act, rows * KB * QB);
  if (e == cudaSuccess) e = dalloc(&h->act_s, rows * KB);
  const size_t counters = h->counters = tile_counters(cfg->max_tokens, cfg->max_tokens < 32 ? cfg->max_tokens : 32, 1, NT, h->num_sms);
  bool wide = false;
  for (int m = 1; m <= cfg->max_tokens && !wide; ++m) wide = linear_granule(*cfg, m, h->num_sms) == 128;
  if (e == cudaSuccess) e = dalloc(&h->parts, part_floats(wide, false, h->num_sms));
  if (e == cudaSuccess) e = dalloc(&h->done, counters);
  if (e == cudaSuccess) e = dalloc(&h->err, 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->done, 0, counters * sizeof(unsigned), st);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->err, 0, sizeof(unsigned), st);
  if (e == cudaSuccess) e = launch_pack_matrix(W, W_s, cfg->N, cfg->K, h->w, h->ws, 1, 0, st);
  // later calls may come on other streams
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    free_linear(h);
    delete h;
    return q_cuda(e, call);
  }
  *out = h;
  return POP_OK;
}

void pop_qlinear_destroy(pop_qlinear_t h) {
  if (!h) return;
  const OnDevice on(h->device);
  cudaDeviceSynchronize();
  free_linear(h);
  delete h;
}

static pop_status linear_check_y(const pop_qlinear* h, int M, const void* x, const void* y, long long ldy,
                                 const char* call) {
  if (M < 0 || M > MAX_ROWS) return q_fail(POP_ERR_INVALID_ARG, call, "M outside [0, 2^27]");
  if (M == 0) return POP_OK;
  if (!x || !y) return q_fail(POP_ERR_INVALID_ARG, call, "NULL x or y");
  if (ldy < h->cfg.N) return q_fail(POP_ERR_INVALID_ARG, call, "ldy < N");
  if (off(y, h->cfg.out_f32 ? 4 : 2)) return q_fail(POP_ERR_INVALID_ARG, call, "y is not aligned to its element");
  return same_device(h->device, call);
}

pop_status pop_qlinear_forward(pop_qlinear_t h, const void* x, long long ldx, int M, void* y, long long ldy,
                               void* stream) {
  const char* call = "pop_qlinear_forward";
  if (!h) return q_fail(POP_ERR_INVALID_ARG, call, "NULL handle");
  const pop_status s = linear_check_y(h, M, x, y, ldy, call);
  if (s != POP_OK || M == 0) return s;
  if (off(x, 16) || ldx < h->cfg.K || ldx % 8)
    return q_fail(POP_ERR_INVALID_ARG, call, "x must be 16-byte aligned, ldx >= K a multiple of 8");
  QRowsArgs in{x, ldx, 0, nullptr, 0, M, h->cfg.K};
  return linear_call(h, in, 2, M, y, ldy, static_cast<cudaStream_t>(stream), call);
}

pop_status pop_qlinear_forward_quantized(pop_qlinear_t h, const void* xq, long long ldq, const float* xs,
                                         long long lds, int M, void* y, long long ldy, void* stream) {
  const char* call = "pop_qlinear_forward_quantized";
  if (!h) return q_fail(POP_ERR_INVALID_ARG, call, "NULL handle");
  const pop_status s = linear_check_y(h, M, xq, y, ldy, call);
  if (s != POP_OK || M == 0) return s;
  if (!xs || off(xs, 4) || lds < qceil(h->cfg.K, QB))
    return q_fail(POP_ERR_INVALID_ARG, call, "xs is NULL or misaligned, or lds < ceil(K / 128)");
  if (off(xq, 8) || ldq < h->cfg.K || ldq % 8)
    return q_fail(POP_ERR_INVALID_ARG, call, "xq must be 8-byte aligned, ldq >= K a multiple of 8");
  QRowsArgs in{xq, ldq, 2, xs, lds, M, h->cfg.K};
  return linear_call(h, in, 1, M, y, ldy, static_cast<cudaStream_t>(stream), call);
}

pop_status pop_qlinear_set_wait_limit(pop_qlinear_t h, uint64_t ns) {
  if (!h || ns == 0) return q_fail(POP_ERR_INVALID_ARG, "pop_qlinear_set_wait_limit", "NULL handle or zero limit");
  h->wait = QWait(ns);
  return POP_OK;
}

pop_status pop_qlinear_check(pop_qlinear_t h) {
  if (!h) return q_fail(POP_ERR_INVALID_ARG, "pop_qlinear_check", "NULL handle");
  if (const pop_status s = same_device(h->device, "pop_qlinear_check"); s != POP_OK) return s;
  return check_word(h->err, h->done, h->counters, "pop_qlinear_check");
}

// -------------------------------------------------------------------------------- experts

pop_status pop_qmoe_create(const pop_qmoe_config* cfg, const void* const* Wg, const void* const* W1,
                           const void* const* W2, const float* const* Sg, const float* const* S1,
                           const float* const* S2, void* stream, pop_qmoe_t* out) {
  const char* call = "pop_qmoe_create";
  const auto bad = [&](const char* why) { return q_fail(POP_ERR_INVALID_ARG, call, why); };
  if (!out) return bad("out is NULL");
  *out = nullptr;
  if (!cfg || !Wg || !W1 || !W2) return bad("NULL argument");
  const bool scaled = Sg || S1 || S2;
  if (scaled && (!Sg || !S1 || !S2)) return bad("Sg, S1 and S2 must all be given or all be NULL");
  if (cfg->n_experts < 1 || cfg->n_experts > POP_QMOE_MAX_EXPERTS) return bad("n_experts out of range");
  if (cfg->top_k < 1 || cfg->top_k > POP_QMOE_MAX_TOP_K) return bad("top_k out of range");
  for (const int d : {cfg->D, cfg->D_FF})
    if (d < 8 || d % 8 || d > POP_QUANT_MAX_DIM) return bad("D and D_FF must be multiples of 8 up to POP_QUANT_MAX_DIM");
  if (cfg->max_tokens < 1 || cfg->max_tokens > (1 << 20)) return bad("max_tokens outside [1, 2^20]");
  if (cfg->out_f32 != 0 && cfg->out_f32 != 1) return bad("out_f32 must be 0 or 1");
  const int E = cfg->n_experts;
  for (int e = 0; e < E; ++e) {
    if (!Wg[e] || !W1[e] || !W2[e] || (scaled && (!Sg[e] || !S1[e] || !S2[e]))) return bad("a NULL matrix or scale");
    if (off(Wg[e], 16) || off(W1[e], 16) || off(W2[e], 16)) return bad("matrices must be 16-byte aligned");
  }
  const pop_status dev = device_supported();
  if (dev != POP_OK) return q_fail(dev, call, "needs an sm_103 device");
  pop_qmoe* m = new (std::nothrow) pop_qmoe();
  if (!m) return q_fail(POP_ERR_OOM, call, "out of host memory");
  m->cfg = *cfg;
  m->device = current_device();
  m->num_sms = sm_count();
  const long long pairs = static_cast<long long>(cfg->max_tokens) * cfg->top_k;
  const long long used = pairs < E ? pairs : E;  // experts that can have rows
  bool wide = false;
  for (int t = 1; t <= cfg->max_tokens && !wide; ++t) wide = qmoe_granule(*cfg, t, m->num_sms) == 128;
  const int most = wide ? 128 : cfg->max_tokens <= 16 ? 16 : cfg->max_tokens <= 32 ? 32 : 64;
  const long long rows = (pairs / most + used) * most;
  const size_t NT = qceil(cfg->D_FF, QB), DT = qceil(cfg->D, QB);
  cudaError_t e = dalloc(&m->wgu, E * NT * DT * 2 * QTILE);
  if (e == cudaSuccess) e = dalloc(&m->wdn, E * DT * NT * QTILE);
  const size_t gu_scales = NT * scale_stride(DT, 2), dn_scales = DT * scale_stride(NT, 1);
  if (e == cudaSuccess) e = dalloc(&m->sgu, E * gu_scales + SCALE_PAD);
  if (e == cudaSuccess) e = dalloc(&m->sdn, E * dn_scales + SCALE_PAD);
  if (e == cudaSuccess) e = dalloc(&m->counts, E);
  if (e == cudaSuccess) e = dalloc(&m->row_of, pairs);
  if (e == cudaSuccess) e = dalloc(&m->act, rows * DT * QB);
  if (e == cudaSuccess) e = dalloc(&m->act_s, rows * DT);
  if (e == cudaSuccess) e = dalloc(&m->h, rows * NT * QB);
  if (e == cudaSuccess) e = dalloc(&m->h_s, rows * NT);
  if (e == cudaSuccess) e = dalloc(&m->o, static_cast<size_t>(rows) * cfg->D);
  const long long few = static_cast<long long>(cfg->max_tokens < 32 ? cfg->max_tokens : 32) * cfg->top_k;
  const size_t counters = m->counters = tile_counters(pairs, few, E, NT > DT ? NT : DT, m->num_sms);
  if (e == cudaSuccess) e = dalloc(&m->parts, part_floats(wide, true, m->num_sms));
  if (e == cudaSuccess) e = dalloc(&m->done, counters);
  if (e == cudaSuccess) e = dalloc(&m->err, 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(m->done, 0, counters * sizeof(unsigned), st);
  if (e == cudaSuccess) e = cudaMemsetAsync(m->err, 0, sizeof(unsigned), st);
  for (int x = 0; x < E && e == cudaSuccess; ++x) {
    uint8_t* gu = m->wgu + x * NT * DT * 2 * QTILE;
    float* sgu = m->sgu + x * gu_scales;
    e = launch_pack_matrix(Wg[x], scaled ? Sg[x] : nullptr, cfg->D_FF, cfg->D, gu, sgu, 2, 0, st);
    if (e == cudaSuccess) e = launch_pack_matrix(W1[x], scaled ? S1[x] : nullptr, cfg->D_FF, cfg->D, gu, sgu, 2, 1, st);
    if (e == cudaSuccess)
      e = launch_pack_matrix(W2[x], scaled ? S2[x] : nullptr, cfg->D, cfg->D_FF, m->wdn + x * DT * NT * QTILE,
                             m->sdn + x * dn_scales, 1, 0, st);
  }
  // later calls may come on other streams
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    free_qmoe(m);
    delete m;
    return q_cuda(e, call);
  }
  *out = m;
  return POP_OK;
}

void pop_qmoe_destroy(pop_qmoe_t m) {
  if (!m) return;
  const OnDevice on(m->device);
  cudaDeviceSynchronize();
  free_qmoe(m);
  delete m;
}

pop_status pop_qmoe_forward(pop_qmoe_t m, const void* x, long long ldx, const int* experts, const float* weights,
                            int T, void* y, long long ldy, void* stream) {
  const char* call = "pop_qmoe_forward";
  const auto bad = [&](const char* why) { return q_fail(POP_ERR_INVALID_ARG, call, why); };
  if (!m) return bad("NULL handle");
  if (T < 0 || T > MAX_ROWS) return bad("T outside [0, 2^27]");
  if (T == 0) return POP_OK;
  if (!x || !experts || !weights || !y) return bad("NULL x, experts, weights or y");
  const pop_qmoe_config& c = m->cfg;
  if (off(x, 16) || ldx < c.D || ldx % 8) return bad("x must be 16-byte aligned, ldx >= D a multiple of 8");
  if (off(y, 16) || ldy < c.D || ldy % (c.out_f32 ? 4 : 8)) return bad("y's rows must be 16-byte aligned, ldy >= D");
  if (off(experts, 4) || off(weights, 4)) return bad("experts or weights is not aligned to its element");
  if (const pop_status s = same_device(m->device, call); s != POP_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t NT = qceil(c.D_FF, QB), DT = qceil(c.D, QB);
  for (int t0 = 0; t0 < T; t0 += c.max_tokens) {
    const int n = T - t0 < c.max_tokens ? T - t0 : c.max_tokens;
    const int pairs = n * c.top_k;
    const int G = qmoe_granule(c, n, m->num_sms);
    const int* ex = experts + static_cast<size_t>(t0) * c.top_k;
    const bool few = pairs <= FEW_PAIRS;
    cudaError_t e = few ? cudaSuccess : launch_plan(ex, pairs, c.n_experts, G, m->counts, m->row_of, m->err, st);
    if (e != cudaSuccess) return q_cuda(e, call);
    QRowsArgs in{static_cast<const uint16_t*>(x) + static_cast<size_t>(t0) * ldx, ldx, 0, nullptr, 0, n, c.D};
    QRowsOut o{};
    o.q = m->act;
    o.s = m->act_s;
    o.G = G;
    o.k = c.top_k;
    if (few) {
      o.experts = ex;
      o.E = c.n_experts;
      o.places = m->row_of;
      o.err = m->err;
    } else {
      o.row_of = m->row_of;
    }
    e = launch_quantize_rows(in, o, st);
    if (e != cudaSuccess) return q_cuda(e, call);
    QGemmArgs g{};
    g.act = m->act;
    g.act_s = m->act_s;
    g.G = G;
    g.w = m->wgu;
    g.ws = m->sgu;
    g.w_stride = NT * DT * 2 * QTILE;
    g.ws_stride = NT * scale_stride(DT, 2);
    g.N = c.D_FF;
    g.K = c.D;
    g.E = c.n_experts;
    g.counts = few ? nullptr : m->counts;
    g.experts = few ? ex : nullptr;
    g.M = pairs;
    g.h = m->h;
    g.h_s = m->h_s;
    g.parts = m->parts;
    g.done = m->done;
    g.err = m->err;
    g.wait = m->wait;
    g.num_sms = m->num_sms;
    e = launch_qgemm(g, true, st);
    if (e != cudaSuccess) return q_cuda(e, call);
    g.act = m->h;
    g.act_s = m->h_s;
    g.w = m->wdn;
    g.ws = m->sdn;
    g.w_stride = NT * DT * QTILE;
    g.ws_stride = DT * scale_stride(NT, 1);
    g.N = c.D;
    g.K = c.D_FF;
    g.h = nullptr;
    g.h_s = nullptr;
    g.y = m->o;
    g.ldy = c.D;
    g.out_f32 = 1;
    e = launch_qgemm(g, false, st);
    if (e != cudaSuccess) return q_cuda(e, call);
    e = launch_combine(m->o, m->row_of, weights + static_cast<size_t>(t0) * c.top_k, n, c.top_k, c.D,
                       static_cast<uint8_t*>(y) + static_cast<size_t>(t0) * ldy * (c.out_f32 ? 4 : 2), ldy, c.out_f32, st);
    if (e != cudaSuccess) return q_cuda(e, call);
  }
  return POP_OK;
}

pop_status pop_qmoe_set_wait_limit(pop_qmoe_t m, uint64_t ns) {
  if (!m || ns == 0) return q_fail(POP_ERR_INVALID_ARG, "pop_qmoe_set_wait_limit", "NULL handle or zero limit");
  m->wait = QWait(ns);
  return POP_OK;
}

pop_status pop_qmoe_check(pop_qmoe_t m) {
  if (!m) return q_fail(POP_ERR_INVALID_ARG, "pop_qmoe_check", "NULL handle");
  if (const pop_status s = same_device(m->device, "pop_qmoe_check"); s != POP_OK) return s;
  return check_word(m->err, m->done, m->counters, "pop_qmoe_check");
}

}  // extern "C"
