// C ABI of the training-step operators declared in include/dion.h: argument
// checks, workspace sizes, and the launches as profiled phases.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "train_checks.h"

using namespace dion;

namespace {

// The forward norm and the codes of plain rows share a kernel and its checks.
int norm_call(const char* name, bool int8_out, NormArgs a, int dtype, int wdtype, hipStream_t stream) {
  Check c;
  c.need(valid_dtype(dtype), "unknown dtype");
  c.need(!a.weight || wdtype == dtype || wdtype == DION_FP32, "the weight must be of x's type or fp32");
  c.need(!a.weight || (std::isfinite(a.eps) && a.eps >= 0.f), "eps must be finite and not negative");
  check_rows(c, a.rows, a.cols, "cols must be positive");
  if (a.cols > kNormMaxCols) c.fail(DION_E_UNSUPPORTED, "more than 65536 columns");
  if (c.code != DION_OK) return c.done();
  const int64_t es = esize(dtype), R = a.rows, C = a.cols;
  const View x{a.x, a.ldx, R, C, es, "x"}, r{a.residual, a.ldr, R, C, es, "residual"},
      w{a.weight, C, 1, C, esize(wdtype), "weight"}, h{a.h, a.ldh, R, C, es, "h"},
      y{a.y, a.ldy, R, C, int8_out ? 1 : es, int8_out ? "q" : "y"}, st{a.stat, 1, R, 1, 4, int8_out ? "scale" : "rstd"};
  check_view(c, x);
  if (a.residual) check_view(c, r);
  if (a.weight) check_view(c, w);
  if (a.h) check_view(c, h);
  check_view(c, y);
  check_view(c, st);
  for (const View& in : {x, r}) {
    check_apart(c, h, in, true);
    check_apart(c, y, in, false);
    check_apart(c, st, in);
  }
  for (const View& out : {h, y, st}) check_apart(c, out, w);
  check_apart(c, h, y);
  check_apart(c, h, st);
  check_apart(c, y, st);
  if (c.code != DION_OK || R == 0) return c.done();
  const double n = (double)R * C;
  return run_phase(name, "dion::k_rmsnorm", 8.0 * n,
                   n * (es * (1 + (a.residual ? 1 : 0) + (a.h ? 1 : 0)) + (int8_out ? 1 : es)), stream,
                   [&]() { launch_rmsnorm(dtype, a.weight ? wdtype : dtype, int8_out, a, stream); });
}

}  // namespace

extern "C" {

int dion_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* h,
                 int64_t ldh, void* y, int64_t ldy, float* rstd, int64_t rows, int32_t cols, int32_t dtype,
                 int32_t weight_dtype, float eps, void* stream) {
  return guarded([&]() {
    if (!weight) return set_error(DION_E_INVAL, "weight is NULL");
    return norm_call("rmsnorm", false, NormArgs{x, residual, weight, h, y, rstd, ldx, ldr, ldh, ldy, rows, cols, eps},
                     dtype, weight_dtype, (hipStream_t)stream);
  });
}

int dion_rmsnorm_int8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* h,
                      int64_t ldh, int8_t* q, int64_t ldq, float* scale, int64_t rows, int32_t cols, int32_t dtype,
                      int32_t weight_dtype, float eps, void* stream) {
  return guarded([&]() {
    if (!weight) return set_error(DION_E_INVAL, "weight is NULL");
    return norm_call("rmsnorm_int8", true,
                     NormArgs{x, residual, weight, h, q, scale, ldx, ldr, ldh, ldq, rows, cols, eps}, dtype,
                     weight_dtype, (hipStream_t)stream);
  });
}

int dion_int8_quantize(const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale, int64_t rows, int32_t cols,
                       int32_t dtype, void* stream) {
  return guarded([&]() {
    return norm_call("int8_quantize", true,
                     NormArgs{x, nullptr, nullptr, nullptr, q, scale, ldx, 0, 0, ldq, rows, cols, 0.f}, dtype, dtype,
                     (hipStream_t)stream);
  });
}

int dion_int8_dequantize(const int8_t* q, int64_t ldq, const float* scale, void* y, int64_t ldy, int64_t rows,
                         int32_t cols, int32_t dtype, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(valid_dtype(dtype), "unknown dtype");
    check_rows(c, rows, cols, "cols must be positive");
    if (c.code != DION_OK) return c.done();
    const View vq{q, ldq, rows, cols, 1, "q"}, vs{scale, 1, rows, 1, 4, "scale"},
        vy{y, ldy, rows, cols, esize(dtype), "y"};
    for (const View& v : {vq, vs, vy}) check_view(c, v);
    check_apart(c, vy, vq);
    check_apart(c, vy, vs);
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    return run_phase("int8_dequantize", "dion::k_int8_dequantize", 0.0, (double)rows * cols * (1 + esize(dtype)), st,
                     [&]() { launch_int8_dequantize(dtype, q, ldq, scale, y, ldy, rows, cols, st); });
  });
}

size_t dion_rmsnorm_backward_workspace_size(int64_t rows, int32_t cols, int32_t dtype) {
  if (rows < 0 || rows > kMaxRows || cols <= 0 || cols > kNormMaxCols || !valid_dtype(dtype)) {
    (void)guarded([&]() { return set_error(DION_E_INVAL, "invalid rows, cols or dtype"); });
    return 0;
  }
  return align256((size_t)norm_back_parts(rows, cols, dtype) * cols * 4 + 1);
}

int dion_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                          const float* rstd, const void* dh, int64_t lddh, void* dx, int64_t lddx, void* dweight,
                          int64_t rows, int32_t cols, int32_t dtype, int32_t weight_dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(valid_dtype(dtype), "unknown dtype");
    c.need(weight_dtype == dtype || weight_dtype == DION_FP32, "the weight must be of x's type or fp32");
    check_rows(c, rows, cols, "cols must be positive");
    if (cols > kNormMaxCols) c.fail(DION_E_UNSUPPORTED, "more than 65536 columns");
    if (c.code != DION_OK) return c.done();
    const int64_t es = esize(dtype), ws = esize(weight_dtype);
    const View vdy{dy, lddy, rows, cols, es, "dy"}, vh{h, ldh, rows, cols, es, "h"},
        vw{weight, cols, 1, cols, ws, "weight"}, vr{rstd, 1, rows, 1, 4, "rstd"},
        vdh{dh, lddh, rows, cols, es, "dh"}, vdx{dx, lddx, rows, cols, es, "dx"},
        vdw{dweight, cols, 1, cols, ws, "dweight"};
    for (const View& v : {vdy, vh, vw, vr, vdx, vdw}) check_view(c, v);
    if (dh) check_view(c, vdh);
    for (const View& in : {vdy, vdh}) check_apart(c, vdx, in, true);
    for (const View& in : {vh, vw, vr, vdw}) check_apart(c, vdx, in);
    for (const View& in : {vdy, vdh, vh, vw, vr}) check_apart(c, vdw, in);
    check_workspace(c, workspace, workspace_bytes, dion_rmsnorm_backward_workspace_size(rows, cols, dtype));
    if (c.code == DION_OK) {
      const View vws{workspace, (int64_t)workspace_bytes, 1, (int64_t)workspace_bytes, 1, "workspace"};
      for (const View& in : {vdy, vdh, vh, vw, vr, vdx, vdw}) check_apart(c, vws, in);
    }
    if (c.code != DION_OK) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    const NormBackArgs a{dy,  h,    weight, rstd, dh,   dx,   dweight, (float*)workspace, lddy, ldh,
                         lddh, lddx, rows,   cols, norm_back_parts(rows, cols, dtype)};
    const double n = (double)rows * cols;
    return run_phase("rmsnorm_backward", "dion::k_rmsnorm_backward", 10.0 * n, n * es * (3 + (dh ? 1 : 0)), st,
                     [&]() { launch_rmsnorm_backward(dtype, weight_dtype, a, st); });
  });
}

size_t dion_int8_linear_workspace_size(const int8_t* a, int64_t lda, const int8_t* b, int64_t ldb, int64_t m,
                                       int64_t n, int32_t k) {
  if (m < 0 || n < 0 || k < 0 || k >= (1 << 17) || m > (1 << 22) || n > (1 << 22)) {
    (void)guarded([&]() { return set_error(DION_E_INVAL, "m, n or k out of range"); });
    return 0;
  }
  if (m == 0 || n == 0) return kNone;
  Int8Args g{};
  g.a = a;
  g.b = b;
  g.lda = lda;
  g.ldb = ldb;
  g.m = m;
  g.n = n;
  g.k = k;
  return reported_size(int8_linear_scratch(g));
}

int dion_int8_linear(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* b, int64_t ldb,
                     const float* b_scale, const void* bias, int32_t bias_dtype, void* out, int64_t ldo, int64_t m,
                     int64_t n, int32_t k, int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() {
    Check c;
    c.need(valid_dtype(out_dtype), "unknown output dtype");
    c.need(!bias || valid_dtype(bias_dtype), "unknown bias dtype");
    c.need(m >= 0 && n >= 0 && k >= 0, "m, n and k must not be negative");
    if (k >= (1 << 17)) c.fail(DION_E_UNSUPPORTED, "k of 2^17 and more may overflow the 32-bit sum");
    if (m > (1 << 22) || n > (1 << 22)) c.fail(DION_E_UNSUPPORTED, "more than 2^22 rows or channels");
    if (c.code != DION_OK) return c.done();
    const View va{a, lda, m, k, 1, "a"}, vb{b, ldb, n, k, 1, "b"}, vsa{a_scale, 1, m, 1, 4, "a_scale"},
        vsb{b_scale, 1, n, 1, 4, "b_scale"}, vbias{bias, n, 1, n, bias ? esize(bias_dtype) : 4, "bias"},
        vo{out, ldo, m, n, esize(out_dtype), "out"};
    for (const View& v : {va, vb, vsa, vsb, vo}) check_view(c, v);
    if (bias) check_view(c, vbias);
    for (const View& in : {va, vb, vsa, vsb, vbias}) check_apart(c, vo, in);
    const size_t need = dion_int8_linear_workspace_size(a, lda, b, ldb, m, n, k);
    if (need > kNone) {
      check_workspace(c, workspace, workspace_bytes, need);
      const View vws{workspace, (int64_t)workspace_bytes, 1, (int64_t)workspace_bytes, 1, "workspace"};
      for (const View& in : {va, vb, vsa, vsb, vbias, vo}) check_apart(c, vws, in);
    }
    if (c.code != DION_OK || m == 0 || n == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    const Int8Args g{a, b, a_scale, b_scale, bias, out, lda, ldb, ldo, m, n, k, bias_dtype, out_dtype,
                     need > kNone ? (int*)workspace : nullptr};
    return run_phase("int8_linear", "dion::k_int8", 2.0 * m * n * k,
                     (double)m * k + (double)n * k + (double)m * n * esize(out_dtype), st,
                     [&]() { launch_int8_linear(g, st); });
  });
}

}  // extern "C"

namespace {

// Checks that the loss and the gradient share.
struct DistillCheck : Check {
  int64_t es = 2;
  View z{}, t{}, ix{}, gl{}, loss{}, stats{}, dz{};
  DistillCheck(const DistillArgs& a, int dtype, int idx_bytes) {
    need(valid_dtype(dtype), "unknown logits dtype");
    need(valid_dtype(a.t_fmt), "unknown teacher dtype");
    need(idx_bytes == 4 || idx_bytes == 8, "teacher indices have 4 or 8 bytes");
    need(std::isfinite(a.temp) && a.temp > 0.f, "temperature must be finite and positive");
    need(a.k >= 0, "k must not be negative");
    check_rows(*this, a.rows, a.vocab, "vocab must be positive");
    if (a.vocab > (1 << 30)) fail(DION_E_UNSUPPORTED, "more than 2^30 logits a row");
    if (a.k > kDistillMaxK) fail(DION_E_UNSUPPORTED, "more than 1024 teacher logits a row");
    if (code != DION_OK) return;
    es = esize(dtype);
    z = View{a.z, a.ldz, a.rows, a.vocab, es, "logits"};
    t = View{a.t, a.k, a.rows, a.k, esize(a.t_fmt), "teacher logits"};
    ix = View{a.idx, a.k, a.rows, a.k, idx_bytes, "teacher indices"};
    gl = View{a.gl, 1, a.rows, 1, 4, "grad_loss"};
    loss = View{a.loss, 1, a.rows, 1, 4, "loss"};
    stats = View{a.stats, 2, a.rows, 2, 4, "stats"};
    dz = View{a.dz, a.ldd, a.rows, a.vocab, es, "dlogits"};
    for (const View& v : {z, t, ix}) check_view(*this, v);
    if (a.gl) check_view(*this, gl);
  }
  // the workspace as the launcher gets it: NULL where none is used, whatever was given
  float2* workspace(void* ws, size_t have, size_t bytes) {
    if (bytes <= kNone) return nullptr;
    check_workspace(*this, ws, have, bytes);
    const View v{ws, (int64_t)have, 1, (int64_t)have, 1, "workspace"};
    for (const View& in : {z, t, ix, gl, loss, stats, dz}) check_apart(*this, v, in);
    return (float2*)ws;
  }
  void output(const View& o, bool in_place = false) {
    check_view(*this, o);
    check_apart(*this, o, z, in_place);
    for (const View& in : {t, ix, gl}) check_apart(*this, o, in);
  }
};

double distill_bytes(const DistillArgs& a, int64_t es, int idx_bytes, bool grad) {
  return (double)a.rows * a.vocab * es * (grad ? 2 : 1) + (double)a.rows * a.k * (esize(a.t_fmt) + idx_bytes);
}

}  // namespace

extern "C" {

size_t dion_distill_topk_workspace_size(int64_t rows, int32_t vocab, int32_t k, int32_t dtype, int32_t gradient) {
  if (rows < 0 || rows > kMaxRows || vocab <= 0 || k < 0 || k > kDistillMaxK || !valid_dtype(dtype)) {
    (void)guarded([&]() { return set_error(DION_E_INVAL, "rows, vocab, k or dtype out of range"); });
    return 0;
  }
  return reported_size(distill_scratch(rows, vocab, k, dtype, gradient != 0));
}

int dion_distill_topk(const void* logits, int64_t ldz, const void* teacher, const void* teacher_idx, float* loss,
                      float* stats, int64_t rows, int32_t vocab, int32_t k, int32_t dtype, int32_t teacher_dtype,
                      int32_t idx_bytes, float temperature, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() {
    DistillArgs a{logits, teacher, teacher_idx, nullptr, loss, (float2*)stats, nullptr, ldz, 0, rows, vocab, k,
                  teacher_dtype, idx_bytes == 8, temperature, nullptr, nullptr, 0};
    DistillCheck c(a, dtype, idx_bytes);
    if (c.code != DION_OK) return c.done();
    c.output(c.loss);
    c.output(c.stats);
    c.need((uintptr_t)stats % 8 == 0, "stats must be 8-byte aligned");
    check_apart(c, c.loss, c.stats);
    a.parts = c.workspace(workspace, workspace_bytes, dion_distill_topk_workspace_size(rows, vocab, k, dtype, 0));
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    return run_phase("distill_topk", "dion::k_distill_forward", 4.0 * rows * vocab,
                     distill_bytes(a, c.es, idx_bytes, false), st, [&]() { launch_distill_forward(dtype, a, st); });
  });
}

int dion_distill_topk_backward(const float* grad_loss, const void* logits, int64_t ldz, const float* stats,
                               const void* teacher, const void* teacher_idx, void* dlogits, int64_t ldd, int64_t rows,
                               int32_t vocab, int32_t k, int32_t dtype, int32_t teacher_dtype, int32_t idx_bytes,
                               float temperature, void* stream) {
  return guarded([&]() {
    const DistillArgs a{logits, teacher, teacher_idx, grad_loss, nullptr, (float2*)stats, dlogits, ldz, ldd, rows,
                        vocab, k, teacher_dtype, idx_bytes == 8, temperature, nullptr, nullptr, 0};
    DistillCheck c(a, dtype, idx_bytes);
    if (c.code != DION_OK) return c.done();
    check_view(c, c.stats);
    c.need((uintptr_t)stats % 8 == 0, "stats must be 8-byte aligned");
    c.output(c.dz, true);
    check_apart(c, c.dz, c.stats);
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    return run_phase("distill_topk_backward", "dion::k_distill_backward", 4.0 * rows * vocab,
                     distill_bytes(a, c.es, idx_bytes, true), st, [&]() { launch_distill_backward(dtype, a, st); });
  });
}

int dion_distill_topk_step(const void* logits, int64_t ldz, const void* teacher, const void* teacher_idx,
                           const float* grad_loss, float* loss, void* dlogits, int64_t ldd, int64_t rows,
                           int32_t vocab, int32_t k, int32_t dtype, int32_t teacher_dtype, int32_t idx_bytes,
                           float temperature, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() {
    DistillArgs a{logits, teacher, teacher_idx, grad_loss, loss, nullptr, dlogits, ldz, ldd, rows,
                  vocab, k, teacher_dtype, idx_bytes == 8, temperature, nullptr, nullptr, 0};
    DistillCheck c(a, dtype, idx_bytes);
    if (c.code != DION_OK) return c.done();
    c.output(c.loss);
    c.output(c.dz, true);
    check_apart(c, c.dz, c.loss);
    a.parts = c.workspace(workspace, workspace_bytes, dion_distill_topk_workspace_size(rows, vocab, k, dtype, 1));
    if (c.code != DION_OK || rows == 0) return c.done();
    const hipStream_t st = (hipStream_t)stream;
    return run_phase("distill_topk_step", "dion::k_distill_step", 8.0 * rows * vocab,
                     distill_bytes(a, c.es, idx_bytes, true), st,
                     [&]() { launch_distill_step(dtype, a, st); });
  });
}

}  // extern "C"
