"""More operators of a training step, beside those of train_ops: layer norms with the residual's addition and their
gradient, microscaled 4-bit floating point (codes, values, product), and the log probabilities of given tokens with
entropy, top alternatives and gradient.

Thin binding over the C ABI (include/dion.h), with the conventions of train_ops: tensors on the current GPU, leading
dimensions that flatten into rows, ``stream``.  A ``stream`` that is given first waits for what the current one holds
(unless it is being captured, when its caller joins the two), so that tensors made there are whole when it reads them;
whoever wants the two to overlap makes it the current one, with ``torch.cuda.stream``, and orders them as needed.
``layer_norm`` and ``log_probs`` are the same operators as torch autograd functions.
"""
from __future__ import annotations

import torch

from ._lib import check, lib
from .train_ops import (_CODE, _F32, _beside, _code, _device, _dense, _fail, _gradient, _handle, _matrix, _new,
                        _new_like, _once, _ptr, _rows, _same, _scratch, _used, _vector, _workspace)


def _behind(stream):
    """a given stream, behind the current one"""
    if stream is None:
        return
    current = torch.cuda.current_stream()
    if stream == current:
        return
    with torch.cuda.stream(stream):
        captured = torch.cuda.is_current_stream_capturing()
    if not captured:
        stream.wait_stream(current)


# ---------------------------------------------------------------- layer norm
def layernorm(x, weight, bias=None, residual=None, eps=1e-5, stream=None):
    """Layer norm of the rows of ``x + residual``: returns (y, h, mean, rstd).

    ``h`` is the sum in x's type, the residual stream carried on (x itself without a residual); ``mean`` and ``rstd``
    (fp32, one for each row) and ``h`` are what ``layernorm_backward`` needs.  ``weight`` and ``bias``: x's type or
    fp32, both the same."""
    dev = _device(x, "x")
    _behind(stream)
    rows, cols, ldx = _matrix(x, "x")
    code = _code(x.dtype, "x")
    ldr = 0 if residual is None else _same(residual, "residual", x, dev)
    _vector(weight, "weight", cols, (x.dtype, torch.float32), dev)
    if bias is not None:
        _vector(bias, "bias", cols, (weight.dtype,), dev)
    y = _new_like(x, x.dtype, stream)
    h = None if residual is None else _new_like(x, x.dtype, stream)
    mean, rstd = _new(x.shape[:-1], torch.float32, x, stream), _new(x.shape[:-1], torch.float32, x, stream)
    rc = lib.dion_layernorm(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), _ptr(bias), _ptr(h), cols,
                            y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(), rows, cols, code,
                            _CODE[weight.dtype], eps, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, x, weight, bias, residual)
    return y, (x if h is None else h), mean, rstd


def layernorm_backward(dy, h, weight, mean, rstd, dh=None, bias=True, workspace=None, stream=None, only_dx=False):
    """Gradients (dx, dweight, dbias) of ``layernorm`` from its ``h``, ``mean`` and ``rstd``; dbias is None without
    ``bias``, and so are both with ``only_dx``, which forms no sums and needs no workspace.

    ``dh`` is the gradient that reaches h itself along the residual stream; dx is the gradient of x and of the residual
    alike."""
    dev = _device(h, "h")
    _behind(stream)
    rows, cols, ldh = _matrix(h, "h")
    code = _code(h.dtype, "h")
    lddy = _same(dy, "dy", h, dev)
    lddh = 0 if dh is None else _same(dh, "dh", h, dev)
    _vector(weight, "weight", cols, (h.dtype, torch.float32), dev)
    _vector(mean, "mean", rows, _F32, dev)
    _vector(rstd, "rstd", rows, _F32, dev)
    if only_dx:
        dx = _new_like(h, h.dtype, stream)
        rc = lib.dion_layernorm_backward_dx(dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), mean.data_ptr(),
                                            rstd.data_ptr(), _ptr(dh), lddh, dx.data_ptr(), cols, rows, cols, code,
                                            _CODE[weight.dtype], _handle(stream, dev))
        if rc:
            check(rc)
        _used(stream, dy, h, weight, mean, rstd, dh)
        return dx, None, None
    keep, ws, have = _workspace(lib.dion_layernorm_backward_workspace_size(rows, cols, code), h, workspace, stream)
    dx = _new_like(h, h.dtype, stream)
    dw = _new_like(weight, weight.dtype, stream)
    db = _new_like(weight, weight.dtype, stream) if bias else None
    rc = lib.dion_layernorm_backward(dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), mean.data_ptr(),
                                     rstd.data_ptr(), _ptr(dh), lddh, dx.data_ptr(), cols, dw.data_ptr(), _ptr(db),
                                     rows, cols, code, _CODE[weight.dtype], ws, have, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, dy, h, weight, mean, rstd, dh, keep)
    return dx, dw, db


# ------------------------------------------- microscaled 4-bit floating point
def _codes(q, scale, what, cols, dev):
    """rows, row strides of codes and scales, and columns of a 4-bit matrix"""
    _beside(scale, "the scales", dev)
    if q.dtype != torch.uint8 or scale.dtype != torch.uint8:
        _fail(f"{what} and its scales must be torch.uint8, got {q.dtype} and {scale.dtype}")
    rows, held, ldq = _matrix(q, what)
    if cols is None:
        cols = 2 * held
    elif (cols + 1) // 2 != held:
        _fail(f"{what}: {held} bytes a row hold {2 * held} or {max(0, 2 * held - 1)} columns, not {cols}")
    srows, blocks, lds = _matrix(scale, "the scales")
    if blocks != (cols + 31) // 32 or srows != rows or q.shape[:-1] != scale.shape[:-1]:
        _fail(f"{what}'s scales: shape {tuple(scale.shape)}, expected {(*q.shape[:-1], (cols + 31) // 32)}")
    return rows, ldq, lds, cols


def mxfp4_quantize(x, stream=None):
    """4-bit floating point codes of the rows of x with a power-of-two scale for each 32 elements: (codes, scale).

    Both uint8: two codes a byte, the even element in the low half, and biased exponents (255 where a block holds an
    infinity or a NaN).  The weights of a product, once; the activations before each."""
    dev = _device(x, "x")
    _behind(stream)
    rows, cols, ldx = _matrix(x, "x")
    code = _code(x.dtype, "x")
    held, blocks = (cols + 1) // 2, (cols + 31) // 32
    q = _new((*x.shape[:-1], held), torch.uint8, x, stream)
    scale = _new((*x.shape[:-1], blocks), torch.uint8, x, stream)
    rc = lib.dion_mxfp4_quantize(x.data_ptr(), ldx, q.data_ptr(), held, scale.data_ptr(), blocks, rows, cols, code,
                                 _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, x)
    return q, scale


def mxfp4_dequantize(q, scale, dtype=torch.bfloat16, cols=None, stream=None):
    """The values that 4-bit codes stand for.  ``cols``: the number of columns where it is odd."""
    dev = _device(q, "q")
    _behind(stream)
    rows, ldq, lds, cols = _codes(q, scale, "q", cols, dev)
    code = _code(dtype, "dtype")
    y = _new((*q.shape[:-1], cols), dtype, q, stream)
    rc = lib.dion_mxfp4_dequantize(q.data_ptr(), ldq, scale.data_ptr(), lds, y.data_ptr(), cols, rows, cols, code,
                                   _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, q, scale)
    return y


def mxfp4_linear(a, a_scale, b, b_scale, bias=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """a (tokens x k) times b (channels x k) transposed, both 4-bit codes with their scales, and an optional bias; the
    products are exact, the sums fp32."""
    dev = _device(a, "a")
    _behind(stream)
    _beside(b, "b", dev)
    m, lda, ldsa, k = _codes(a, a_scale, "a", None, dev)
    n, ldb, ldsb, kb = _codes(b, b_scale, "b", None, dev)
    if b.dim() != 2 or kb != k:
        _fail(f"b: shape {tuple(b.shape)}, expected (channels, {k // 2})")
    code = _code(out_dtype, "out_dtype")
    if bias is not None:
        _vector(bias, "bias", n, _CODE, dev)
    pa, psa, pb, psb = a.data_ptr(), a_scale.data_ptr(), b.data_ptr(), b_scale.data_ptr()
    need = lib.dion_mxfp4_linear_workspace_size(pa, lda, psa, ldsa, pb, ldb, psb, ldsb, m, n, k)
    keep, ws, have = _scratch(need, a, workspace, stream)
    out = _new((*a.shape[:-1], n), out_dtype, a, stream)
    rc = lib.dion_mxfp4_linear(pa, lda, psa, ldsa, pb, ldb, psb, ldsb, _ptr(bias),
                               0 if bias is None else _CODE[bias.dtype], out.data_ptr(), n, m, n, k, code, ws, have,
                               _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, a, a_scale, b, b_scale, bias, keep)
    return out


# ----------------------------------------------------------- log probabilities
def _logprob_inputs(logits, tokens, stream):
    dev = _device(logits, "logits")
    _behind(stream)
    rows, vocab, ldz = _matrix(logits, "logits")
    code = _code(logits.dtype, "logits")
    if tokens is None:
        return dev, rows, vocab, ldz, code, None, 8
    _beside(tokens, "tokens", dev)
    if tokens.shape != logits.shape[:-1]:
        _fail(f"tokens: shape {tuple(tokens.shape)}, expected {tuple(logits.shape[:-1])}")
    if tokens.dtype not in (torch.int64, torch.int32):
        _fail(f"tokens: unsupported dtype {tokens.dtype}")
    return dev, rows, vocab, ldz, code, _dense(tokens, stream), tokens.element_size()


def token_logprobs(logits, tokens, temperature=1.0, workspace=None, stream=None):
    """Log probability of each row's token and the row's entropy: returns (logprob, entropy, stats).

    ``logits``: rows x vocab; ``tokens`` (int64 or int32): rows.  A token outside the vocabulary (padding) has
    logprob 0.  ``stats`` is for ``token_logprobs_backward``."""
    dev, rows, vocab, ldz, code, tok, tb = _logprob_inputs(logits, tokens, stream)
    if tok is None:
        _fail("tokens are needed")
    keep, ws, have = _scratch(lib.dion_token_logprobs_workspace_size(rows, vocab, 0, code), logits, workspace, stream)
    shape = logits.shape[:-1]
    logprob, entropy = _new(shape, torch.float32, logits, stream), _new(shape, torch.float32, logits, stream)
    stats = _new((*shape, 4), torch.float32, logits, stream)
    rc = lib.dion_token_logprobs(logits.data_ptr(), ldz, tok.data_ptr(), logprob.data_ptr(), entropy.data_ptr(),
                                 stats.data_ptr(), None, None, rows, vocab, 0, code, tb, temperature, ws, have,
                                 _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, logits, tok, keep)
    return logprob, entropy, stats


def top_logprobs(logits, k, tokens=None, temperature=1.0, workspace=None, stream=None):
    """The k likeliest tokens of each row: returns (top, index, logprob, entropy).

    ``top`` (fp32, descending) and ``index`` (int64; equal logits in the order of their index) have k places a row;
    places beyond the logits above -inf hold -inf and -1, which ``distill_loss`` takes as absent entries.  ``logprob``
    is that of ``tokens`` as in ``token_logprobs``, None without them."""
    dev, rows, vocab, ldz, code, tok, tb = _logprob_inputs(logits, tokens, stream)
    keep, ws, have = _scratch(lib.dion_token_logprobs_workspace_size(rows, vocab, k, code), logits, workspace, stream)
    shape = logits.shape[:-1]
    logprob = None if tok is None else _new(shape, torch.float32, logits, stream)
    entropy = _new(shape, torch.float32, logits, stream)
    top, index = _new((*shape, k), torch.float32, logits, stream), _new((*shape, k), torch.int64, logits, stream)
    rc = lib.dion_token_logprobs(logits.data_ptr(), ldz, _ptr(tok), _ptr(logprob), entropy.data_ptr(), None,
                                 top.data_ptr(), index.data_ptr(), rows, vocab, k, code, tb, temperature, ws, have,
                                 _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, logits, tok, keep)
    return top, index, logprob, entropy


def token_logprobs_backward(grad_logprob, grad_entropy, logits, stats, tokens, temperature=1.0, out=None, stream=None):
    """Gradient of the logits from ``token_logprobs``'s stats and the gradients of each row's log probability and
    entropy (None: 0).  ``out`` may be the logits themselves."""
    dev, rows, vocab, ldz, code, tok, tb = _logprob_inputs(logits, tokens, stream)
    for g, what in ((grad_logprob, "grad_logprob"), (grad_entropy, "grad_entropy")):
        if g is not None:
            _vector(g, what, rows, _F32, dev)
    _vector(stats, "stats", 4 * rows, _F32, dev)
    out, ldd = _gradient(logits, rows, vocab, out, stream, dev)
    rc = lib.dion_token_logprobs_backward(_ptr(grad_logprob), _ptr(grad_entropy), logits.data_ptr(), ldz,
                                          stats.data_ptr(), _ptr(tok), out.data_ptr(), ldd, rows, vocab, code, tb,
                                          temperature, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, grad_logprob, grad_entropy, logits, stats, tok, out)
    return out


# ------------------------------------------------------------------- autograd
class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps):
        y, h, mean, rstd = layernorm(x, weight, bias, residual, eps)
        ctx.save_for_backward(h, weight, mean, rstd)
        ctx.residual, ctx.bias = residual is not None, bias is not None
        ctx.set_materialize_grads(False)   # an output that nothing used sends None, not zeros to be read
        return (y, h) if ctx.residual else y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, mean, rstd = ctx.saved_tensors
        if dy is None:
            return dh, None, None, dh, None
        w, b = ctx.needs_input_grad[1], ctx.bias and ctx.needs_input_grad[2]   # frozen ones have no sums formed

        def gradients(dy, h, weight, dh):
            return layernorm_backward(dy.contiguous(), h, weight, mean, rstd, None if dh is None else dh.contiguous(),
                                      bias=b, only_dx=not (w or b))

        dx, dw, db = _once(gradients, dy, h, weight, dh)
        return dx, (dw if w else None), db, (dx if ctx.residual else None), None


def layer_norm(x, weight, bias=None, residual=None, eps=1e-5):
    """``layernorm`` for automatic differentiation, once: returns y, or (y, h) with a residual.
    Tensors of any strides; what does not lie in rows is copied first."""
    return _LayerNorm.apply(_rows(x), _rows(weight), _rows(bias), _rows(residual), eps)


class _LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature):
        logprob, entropy, stats = token_logprobs(logits, tokens, temperature)
        ctx.save_for_backward(logits, stats, tokens)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        return logprob, entropy

    @staticmethod
    def backward(ctx, gl, ge):
        if gl is None and ge is None:
            return None, None, None
        logits, stats, tokens = ctx.saved_tensors

        def gradient(gl, ge, logits):
            dense = lambda g: None if g is None else g.contiguous()
            return token_logprobs_backward(dense(gl), dense(ge), logits, stats, tokens, ctx.temperature)

        return _once(gradient, gl, ge, logits), None, None


def log_probs(logits, tokens, temperature=1.0):
    """``token_logprobs`` for automatic differentiation, once: returns (logprob, entropy) of each row.
    Tensors of any strides, as for ``layer_norm``."""
    return _LogProbs.apply(_rows(logits), tokens, temperature)
