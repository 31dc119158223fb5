// C ABI of the layer norm, the microscaled 4-bit operators and the log
// probabilities declared in include/dion.h: argument checks, workspace sizes,
// and the launches as profiled phases.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <string>

#include "model_internal.h"
#include "train_checks.h"

using namespace dion;

namespace {

// The gradient with (sums) and without those of the weight and the bias.
int layernorm_backward_call(LayerNormBackArgs a, bool sums, int32_t dtype, int32_t weight_dtype, size_t workspace_bytes,
                            hipStream_t st) {
  Check c;
  const int64_t rows = a.rows;
  const int32_t cols = a.cols;
  c.need(valid_dtype(dtype), "unknown dtype");
  c.need(weight_dtype == dtype || weight_dtype == DION_FP32, "the weight must be of x's type or fp32");
  check_rows(c, rows, cols, "cols must be positive");
  if (cols > kLayerNormMaxCols) c.fail(DION_E_UNSUPPORTED, "more than 65536 columns");
  if (c.code != DION_OK) return c.done();
  const int64_t es = esize(dtype), ws = esize(weight_dtype);
  const View vdy{a.dy, a.lddy, rows, cols, es, "dy"}, vh{a.h, a.ldh, rows, cols, es, "h"},
      vw{a.weight, cols, 1, cols, ws, "weight"}, vm{a.mean, 1, rows, 1, 4, "mean"}, vr{a.rstd, 1, rows, 1, 4, "rstd"},
      vdh{a.dh, a.lddh, rows, cols, es, "dh"}, vdx{a.dx, a.lddx, rows, cols, es, "dx"},
      vdw{a.dweight, cols, 1, cols, ws, "dweight"}, vdb{a.dbias, cols, 1, cols, ws, "dbias"};
  for (const View& v : {vdy, vh, vw, vm, vr, vdx}) check_view(c, v);
  if (sums) check_view(c, vdw);
  if (a.dh) check_view(c, vdh);
  if (a.dbias) check_view(c, vdb);
  for (const View& in : {vdy, vdh}) check_apart(c, vdx, in, true);
  for (const View& in : {vh, vw, vm, vr, vdw, vdb}) check_apart(c, vdx, in);
  for (const View& out : {vdw, vdb})
    for (const View& in : {vdy, vdh, vh, vw, vm, vr}) check_apart(c, out, in);
  check_apart(c, vdw, vdb);
  if (sums) {
    check_workspace(c, a.partial, workspace_bytes, dion_layernorm_backward_workspace_size(rows, cols, dtype));
    if (c.code == DION_OK) {
      const View vws{a.partial, (int64_t)workspace_bytes, 1, (int64_t)workspace_bytes, 1, "workspace"};
      for (const View& in : {vdy, vdh, vh, vw, vm, vr, vdx, vdw, vdb}) check_apart(c, vws, in);
    }
  }
  if (c.code != DION_OK || (rows == 0 && !sums)) return c.done();
  a.parts = layernorm_back_parts(rows, cols, dtype);
  const double n = (double)rows * cols;
  return run_phase("layernorm_backward", "dion::k_layernorm_backward", 14.0 * n, n * es * (3 + (a.dh ? 1 : 0)), st,
                   [&]() { launch_layernorm_backward(dtype, weight_dtype, a, st); });
}

}  // namespace

extern "C" {

int dion_layernorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, const void* bias,
                   void* h, int64_t ldh, void* y, int64_t ldy, float* mean, float* rstd, int64_t rows, int32_t cols,
                   int32_t dtype, int32_t weight_dtype, float eps, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(weight, "weight is NULL");
    c.need(valid_dtype(dtype), "unknown dtype");
    c.need(weight_dtype == dtype || weight_dtype == DION_FP32, "weight and bias must be of x's type or fp32");
    c.need(std::isfinite(eps) && eps >= 0.f, "eps must be finite and not negative");
    check_rows(c, rows, cols, "cols must be positive");
    if (cols > kLayerNormMaxCols) c.fail(DION_E_UNSUPPORTED, "more than 65536 columns");
    if (c.code != DION_OK) return c.done();
    const int64_t es = esize(dtype), ws = esize(weight_dtype);
    const View vx{x, ldx, rows, cols, es, "x"}, vr{residual, ldr, rows, cols, es, "residual"},
        vw{weight, cols, 1, cols, ws, "weight"}, vb{bias, cols, 1, cols, ws, "bias"}, vh{h, ldh, rows, cols, es, "h"},
        vy{y, ldy, rows, cols, es, "y"}, vm{mean, 1, rows, 1, 4, "mean"}, vs{rstd, 1, rows, 1, 4, "rstd"};
    for (const View& v : {vx, vw, vy, vm, vs}) check_view(c, v);
    if (residual) check_view(c, vr);
    if (bias) check_view(c, vb);
    if (h) check_view(c, vh);
    for (const View& in : {vx, vr}) {
      check_apart(c, vh, in, true);
      for (const View& out : {vy, vm, vs}) check_apart(c, out, in);
    }
    for (const View& out : {vh, vy, vm, vs})
      for (const View& in : {vw, vb}) check_apart(c, out, in);
    for (const View& out : {vy, vm, vs}) check_apart(c, out, vh);
    for (const View& out : {vm, vs}) check_apart(c, out, vy);
    check_apart(c, vm, vs);
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    const LayerNormArgs a{x, residual, weight, bias, h, y, mean, rstd, ldx, ldr, ldh, ldy, rows, cols, eps};
    const double n = (double)rows * cols;
    return run_phase("layernorm", "dion::k_layernorm", 9.0 * n, n * es * (2 + (residual ? 1 : 0) + (h ? 1 : 0)), st,
                     [&]() { launch_layernorm(dtype, weight_dtype, a, st); });
  });
}

size_t dion_layernorm_backward_workspace_size(int64_t rows, int32_t cols, int32_t dtype) {
  if (rows < 0 || rows > kMaxRows || cols <= 0 || cols > kLayerNormMaxCols || !valid_dtype(dtype)) {
    (void)guarded([&]() { return set_error(DION_E_INVAL, "invalid rows, cols or dtype"); });
    return 0;
  }
  return align256((size_t)layernorm_back_parts(rows, cols, dtype) * cols * 8 + 1);
}

int dion_layernorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                            const float* mean, const float* rstd, const void* dh, int64_t lddh, void* dx, int64_t lddx,
                            void* dweight, void* dbias, int64_t rows, int32_t cols, int32_t dtype, int32_t weight_dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() {
    const LayerNormBackArgs a{dy,   h,   weight, mean, rstd, dh,   dx, dweight, dbias, (float*)workspace,
                              lddy, ldh, lddh,   lddx, rows, cols, 0};
    return layernorm_backward_call(a, true, dtype, weight_dtype, workspace_bytes, (hipStream_t)stream);
  });
}

int dion_layernorm_backward_dx(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                               const float* mean, const float* rstd, const void* dh, int64_t lddh, void* dx,
                               int64_t lddx, int64_t rows, int32_t cols, int32_t dtype, int32_t weight_dtype,
                               void* stream) {
  return guarded([&]() {
    const LayerNormBackArgs a{dy,   h,   weight, mean, rstd, dh,   dx, nullptr, nullptr, nullptr,
                              lddy, ldh, lddh,   lddx, rows, cols, 0};
    return layernorm_backward_call(a, false, dtype, weight_dtype, 0, (hipStream_t)stream);
  });
}

}  // extern "C"

namespace {

// Codes and scales of a matrix of rows x cols.
struct MxViews {
  View q, s;
  MxViews(const void* q_, int64_t ldq, const void* s_, int64_t lds, int64_t rows, int64_t cols, const char* codes,
          const char* scales)
      : q{q_, ldq, rows, (cols + 1) / 2, 1, codes}, s{s_, lds, rows, (cols + 31) / 32, 1, scales} {}
};

constexpr int32_t kMxMaxK = 1 << 22, kMxMaxCols = 1 << 30;
constexpr int64_t kMxMaxRows = 1 << 22;

}  // namespace

extern "C" {

int dion_mxfp4_quantize(const void* x, int64_t ldx, uint8_t* q, int64_t ldq, uint8_t* scale, int64_t lds, int64_t rows,
                        int32_t cols, int32_t dtype, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(valid_dtype(dtype), "unknown dtype");
    check_rows(c, rows, cols, "cols must be positive");
    if (cols > kMxMaxCols) c.fail(DION_E_UNSUPPORTED, "more than 2^30 columns");
    if (c.code != DION_OK) return c.done();
    const View vx{x, ldx, rows, cols, esize(dtype), "x"};
    const MxViews v(q, ldq, scale, lds, rows, cols, "q", "scale");
    for (const View& w : {vx, v.q, v.s}) check_view(c, w);
    check_apart(c, v.q, vx);
    check_apart(c, v.s, vx);
    check_apart(c, v.q, v.s);
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    const MxCodesArgs a{(void*)x, q, scale, ldx, ldq, lds, rows, cols};
    const double n = (double)rows * cols;
    return run_phase("mxfp4_quantize", "dion::k_mxfp4_quantize", 4.0 * n, n * (esize(dtype) + 17.0 / 32), st,
                     [&]() { launch_mxfp4_quantize(dtype, a, st); });
  });
}

int dion_mxfp4_dequantize(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds, void* y, int64_t ldy,
                          int64_t rows, int32_t cols, int32_t dtype, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(valid_dtype(dtype), "unknown dtype");
    check_rows(c, rows, cols, "cols must be positive");
    if (cols > kMxMaxCols) c.fail(DION_E_UNSUPPORTED, "more than 2^30 columns");
    if (c.code != DION_OK) return c.done();
    const View vy{y, ldy, rows, cols, esize(dtype), "y"};
    const MxViews v(q, ldq, scale, lds, rows, cols, "q", "scale");
    for (const View& w : {vy, v.q, v.s}) check_view(c, w);
    check_apart(c, vy, v.q);
    check_apart(c, vy, v.s);
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    const MxCodesArgs a{y, (uint8_t*)q, (uint8_t*)scale, ldy, ldq, lds, rows, cols};
    const double n = (double)rows * cols;
    return run_phase("mxfp4_dequantize", "dion::k_mxfp4_dequantize", 0.0, n * (esize(dtype) + 17.0 / 32), st,
                     [&]() { launch_mxfp4_dequantize(dtype, a, st); });
  });
}

size_t dion_mxfp4_linear_workspace_size(const uint8_t* a, int64_t lda, const uint8_t* a_scale, int64_t ldsa,
                                        const uint8_t* b, int64_t ldb, const uint8_t* b_scale, int64_t ldsb, int64_t m,
                                        int64_t n, int32_t k) {
  if (m < 0 || n < 0 || k < 0 || k % 2 || k > kMxMaxK || m > kMxMaxRows || n > kMxMaxRows) {
    (void)guarded([&]() { return set_error(DION_E_INVAL, "m, n or k out of range, or k odd"); });
    return 0;
  }
  if (m == 0 || n == 0) return kNone;
  MxArgs g{};
  g.a = a;
  g.sa = a_scale;
  g.b = b;
  g.sb = b_scale;
  g.lda = lda;
  g.ldsa = ldsa;
  g.ldb = ldb;
  g.ldsb = ldsb;
  g.m = m;
  g.n = n;
  g.kb = k / 2;
  return reported_size(mxfp4_linear_scratch(g));
}

int dion_mxfp4_linear(const uint8_t* a, int64_t lda, const uint8_t* a_scale, int64_t ldsa, const uint8_t* b,
                      int64_t ldb, const uint8_t* b_scale, int64_t ldsb, const void* bias, int32_t bias_dtype,
                      void* out, int64_t ldo, int64_t m, int64_t n, int32_t k, int32_t out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(valid_dtype(out_dtype), "unknown output dtype");
    c.need(!bias || valid_dtype(bias_dtype), "unknown bias dtype");
    c.need(m >= 0 && n >= 0 && k >= 0, "m, n and k must not be negative");
    c.need(k % 2 == 0, "k must be even: codes lie two to a byte");
    if (k > kMxMaxK) c.fail(DION_E_UNSUPPORTED, "k of more than 2^22");
    if (m > kMxMaxRows || n > kMxMaxRows) c.fail(DION_E_UNSUPPORTED, "more than 2^22 rows or channels");
    if (c.code != DION_OK) return c.done();
    const MxViews va(a, lda, a_scale, ldsa, m, k, "a", "a_scale"), vb(b, ldb, b_scale, ldsb, n, k, "b", "b_scale");
    const View vbias{bias, n, 1, n, bias ? esize(bias_dtype) : 4, "bias"}, vo{out, ldo, m, n, esize(out_dtype), "out"};
    for (const View& v : {va.q, va.s, vb.q, vb.s, vo}) check_view(c, v);
    if (bias) check_view(c, vbias);
    for (const View& in : {va.q, va.s, vb.q, vb.s, vbias}) check_apart(c, vo, in);
    const size_t need = c.code != DION_OK ? 0 : dion_mxfp4_linear_workspace_size(a, lda, a_scale, ldsa, b, ldb, b_scale, ldsb, m, n, k);
    if (need > kNone) {
      check_workspace(c, workspace, workspace_bytes, need);
      const View vws{workspace, (int64_t)workspace_bytes, 1, (int64_t)workspace_bytes, 1, "workspace"};
      for (const View& in : {va.q, va.s, vb.q, vb.s, vbias, vo}) check_apart(c, vws, in);
    }
    if (c.code != DION_OK || m == 0 || n == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    const MxArgs g{a,    a_scale, b,    b_scale, bias, out,   lda,        ldsa,      ldb,
                   ldsb, ldo,     m,    n,       k / 2, bias_dtype, out_dtype, need > kNone ? (float*)workspace : nullptr};
    return run_phase("mxfp4_linear", "dion::k_mxfp4", 2.0 * m * n * k,
                     ((double)m + n) * k * 17 / 32 + (double)m * n * esize(out_dtype), st,
                     [&]() { launch_mxfp4_linear(g, st); });
  });
}

}  // extern "C"

namespace {

// Checks that the log probabilities and their gradient share.
struct LogprobCheck : Check {
  int64_t es = 2;
  View z{}, tok{};
  LogprobCheck(const LogprobArgs& a, int dtype, int tok_bytes) {
    need(valid_dtype(dtype), "unknown logits dtype");
    need(!a.tok || tok_bytes == 4 || tok_bytes == 8, "tokens have 4 or 8 bytes");
    need(std::isfinite(a.temp) && a.temp >= FLT_MIN, "temperature must be finite and 2^-126 at least");   // 1 / T is finite
    check_rows(*this, a.rows, a.vocab, "vocab must be positive");
    if (a.vocab > (1 << 30)) fail(DION_E_UNSUPPORTED, "more than 2^30 logits a row");
    if (code != DION_OK) return;
    es = esize(dtype);
    z = View{a.z, a.ldz, a.rows, a.vocab, es, "logits"};
    tok = View{a.tok, 1, a.rows, 1, a.tok ? tok_bytes : 8, "tokens"};
    check_view(*this, z);
    if (a.tok) check_view(*this, tok);
  }
};

}  // namespace

extern "C" {

size_t dion_token_logprobs_workspace_size(int64_t rows, int32_t vocab, int32_t top, int32_t dtype) {
  if (rows < 0 || rows > kMaxRows || vocab <= 0 || vocab > (1 << 30) || top < 0 || top > kLogprobMaxTop ||
      (top > 0 && vocab > kLogprobMaxTopVocab) || !valid_dtype(dtype)) {
    (void)guarded([&]() { return set_error(DION_E_INVAL, "rows, vocab, top or dtype out of range"); });
    return 0;
  }
  return reported_size(logprob_scratch(rows, vocab, top, dtype));
}

int dion_token_logprobs(const void* logits, int64_t ldz, const void* tokens, float* logprob, float* entropy,
                        float* stats, float* top_logprob, int64_t* top_index, int64_t rows, int32_t vocab, int32_t top,
                        int32_t dtype, int32_t token_bytes, float temperature, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return guarded([&]() {
    LogprobArgs a{};
    a.z = logits;
    a.tok = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.stats = (float4*)stats;
    a.top = top_logprob;
    a.index = top_index;
    a.ldz = ldz;
    a.rows = rows;
    a.vocab = vocab;
    a.k = top;
    a.tok64 = token_bytes == 8;
    a.temp = temperature;
    LogprobCheck c(a, dtype, token_bytes);
    c.need(top >= 0, "top must not be negative");
    if (top > kLogprobMaxTop) c.fail(DION_E_UNSUPPORTED, "more than 1024 alternatives");
    if (top > 0 && vocab > kLogprobMaxTopVocab) c.fail(DION_E_UNSUPPORTED, "alternatives among more than 2^19 logits");
    if (c.code != DION_OK) return c.done();
    const View vl{logprob, 1, rows, 1, 4, "logprob"}, ve{entropy, 1, rows, 1, 4, "entropy"},
        vs{stats, 4, rows, 4, 4, "stats"}, vt{top_logprob, top, rows, top, 4, "top_logprob"},
        vi{top_index, top, rows, top, 8, "top_index"};
    if (tokens) check_view(c, vl);
    for (const View& v : {ve, vt, vi}) check_view(c, v);
    if (stats) check_view(c, vs);
    c.need((uintptr_t)stats % 16 == 0, "stats must be 16-byte aligned");
    const View out[] = {vl, ve, vs, vt, vi};
    for (int i = 0; i < 5; ++i) {
      check_apart(c, out[i], c.z);
      check_apart(c, out[i], c.tok);
      for (int j = 0; j < i; ++j) check_apart(c, out[i], out[j]);
    }
    const size_t need = c.code != DION_OK ? 0 : dion_token_logprobs_workspace_size(rows, vocab, top, dtype);
    if (need > kNone) {
      check_workspace(c, workspace, workspace_bytes, need);
      const View vws{workspace, (int64_t)workspace_bytes, 1, (int64_t)workspace_bytes, 1, "workspace"};
      for (const View& v : out) check_apart(c, vws, v);
      check_apart(c, vws, c.z);
      check_apart(c, vws, c.tok);
      a.parts = (float4*)workspace;
    }
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    return run_phase("token_logprobs", "dion::k_logprobs", 6.0 * rows * vocab,
                     (double)rows * vocab * c.es + 12.0 * rows * top, st, [&]() { launch_token_logprobs(dtype, a, st); });
  });
}

int dion_token_logprobs_backward(const float* grad_logprob, const float* grad_entropy, const void* logits, int64_t ldz,
                                 const float* stats, const void* tokens, void* dlogits, int64_t ldd, int64_t rows,
                                 int32_t vocab, int32_t dtype, int32_t token_bytes, float temperature, void* stream) {
  return guarded([&]() {
    LogprobArgs a{};
    a.z = logits;
    a.tok = tokens;
    a.stats = (float4*)stats;
    a.gl = grad_logprob;
    a.ge = grad_entropy;
    a.dz = dlogits;
    a.ldz = ldz;
    a.ldd = ldd;
    a.rows = rows;
    a.vocab = vocab;
    a.tok64 = token_bytes == 8;
    a.temp = temperature;
    LogprobCheck c(a, dtype, token_bytes);
    if (c.code != DION_OK) return c.done();
    const View vl{grad_logprob, 1, rows, 1, 4, "grad_logprob"}, ve{grad_entropy, 1, rows, 1, 4, "grad_entropy"},
        vs{stats, 4, rows, 4, 4, "stats"}, vd{dlogits, ldd, rows, vocab, c.es, "dlogits"};
    if (grad_logprob) check_view(c, vl);
    if (grad_entropy) check_view(c, ve);
    check_view(c, vs);
    c.need((uintptr_t)stats % 16 == 0, "stats must be 16-byte aligned");
    check_view(c, vd);
    check_apart(c, vd, c.z, true);
    for (const View& in : {c.tok, vl, ve, vs}) check_apart(c, vd, in);
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    return run_phase("token_logprobs_backward", "dion::k_logprobs_backward", 8.0 * rows * vocab,
                     2.0 * rows * vocab * c.es, st, [&]() { launch_token_logprobs_backward(dtype, a, st); });
  });
}

}  // extern "C"
