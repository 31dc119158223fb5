"""The operators of a training step around the optimizer: RMS norms with the
residual's addition (16-bit, fp32 or 8-bit output, and the gradient), the
product of 8-bit integers with scales for tokens and channels, and the
distillation loss on a teacher's top logits with its gradient.

Thin binding over the C ABI (include/dion.h): it checks tensors, allocates the
outputs and passes pointers; the arithmetic runs in libdion.so.  ``rms_norm``
and ``distill_loss`` are the same operators as torch autograd functions.

Tensors are on the current GPU.  Matrices may have leading dimensions that
flatten into rows and rows further apart than they are long (a padded
vocabulary, a slice of columns); the elements of a row are contiguous.  With
``stream`` the work runs there, outputs and workspaces are allocated for it,
and every tensor is recorded as used by it.
"""
from __future__ import annotations

import torch

from ._lib import DION_BF16, DION_FP16, DION_FP32, DionError, check, lib

_CODE = {torch.bfloat16: DION_BF16, torch.float32: DION_FP32, torch.float16: DION_FP16}


def _fail(msg):
    raise DionError(-1, msg)


def _code(dtype, what):
    code = _CODE.get(dtype)
    if code is None:
        _fail(f"{what}: unsupported dtype {dtype}")
    return code


# the handle of a device's current stream, without a Stream object around it
# (0.1 against 2.7 us, of a call that takes about 10 on the host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(t, what):
    """the tensor's device, which has to be the current one"""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{what} must be a tensor on the GPU")
    dev = t.get_device()
    if dev != _current_device():
        _fail(f"{what} is on another device than the current one")
    return dev


def _beside(t, what, dev):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _fail(f"{what} must be a tensor on the same GPU as the others")


def _matrix(t, what):
    """rows, cols and row stride of a tensor whose leading dimensions flatten into rows"""
    shape = t.shape
    if len(shape) == 2 and t.is_contiguous():
        rows, cols = shape
        return rows, cols, cols
    if len(shape) != 2:
        if len(shape) == 0:
            _fail(f"{what} must have at least one dimension")
        try:
            t = t.view(-1, shape[-1]) if t.numel() else t.reshape(shape[:-1].numel(), shape[-1])
        except RuntimeError:
            _fail(f"{what}: the leading dimensions do not flatten into equally spaced rows")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1 and rows > 0:
        _fail(f"{what}: the elements of a row must be contiguous")
    return rows, cols, (t.stride(0) if rows > 1 else cols)


def _same(t, what, like, dev):
    """row stride of a tensor that has to match another's shape and dtype"""
    _beside(t, what, dev)
    if t.shape != like.shape:
        _fail(f"{what}: shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    if t.dtype != like.dtype:
        _fail(f"{what}: expected {like.dtype}, got {t.dtype}")
    return _matrix(t, what)[2]


def _vector(t, what, n, dtypes, dev):
    _beside(t, what, dev)
    if t.numel() != n or (n > 1 and not t.is_contiguous()):
        _fail(f"{what} must be contiguous with {n} entries")
    if t.dtype not in dtypes:
        _fail(f"{what}: unsupported dtype {t.dtype}")


def _handle(stream, dev):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _new(shape, dtype, like, stream):
    """A tensor for a call on `stream`: allocated in that stream's memory, and
    known to be used by the current one, which reads the results."""
    if stream is None:   # (a bare length takes torch 0.4 us less than a shape)
        return torch.empty(shape if len(shape) != 1 else shape[0], dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=like.device)
    out.record_stream(torch.cuda.current_stream())
    return out


def _new_like(like, dtype, stream):
    """the same with another tensor's shape, contiguous"""
    if stream is None and like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return _new(like.shape, dtype, like, stream)


def _workspace(nbytes, like, given, stream):
    """the caller's workspace, or a new one, with its aligned address and length"""
    if nbytes == 0:
        raise DionError(-1, lib.dion_last_error().decode())
    if given is None:
        given = _new((nbytes + 256,), torch.uint8, like, stream)
    elif not given.is_cuda or not given.is_contiguous():
        _fail("the workspace must be a contiguous tensor on the GPU")
    at = given.data_ptr()
    off = -at % 256
    have = given.numel() * given.element_size() - off
    if have < nbytes:
        raise DionError(-3, f"workspace too small: need {nbytes} bytes")
    return given, at + off, have


def _scratch(nbytes, like, given, stream):
    """the same where a size of 256 means that the call uses none"""
    if nbytes == 256 and given is None:
        return None, None, 0
    return _workspace(nbytes, like, given, stream)


def _used(stream, *tensors):
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


_F32 = (torch.float32,)


# ------------------------------------------------------------------ RMS norm
def _norm_inputs(x, weight, residual):
    dev = _device(x, "x")
    rows, cols, ldx = _matrix(x, "x")
    code = _code(x.dtype, "x")
    ldr = 0 if residual is None else _same(residual, "residual", x, dev)
    _vector(weight, "weight", cols, (x.dtype, torch.float32), dev)
    return dev, rows, cols, ldx, ldr, code, _CODE[weight.dtype]


def rmsnorm(x, weight, residual=None, eps=1e-6, stream=None):
    """RMS norm of the rows of ``x + residual``: returns (y, h, rstd).

    ``h`` is the sum in x's type, the residual stream carried on (x itself
    without a residual); ``rstd`` (fp32, one for each row) and ``h`` are what
    ``rmsnorm_backward`` needs.  ``weight``: x's type or fp32."""
    dev, rows, cols, ldx, ldr, code, wcode = _norm_inputs(x, weight, residual)
    y = _new_like(x, x.dtype, stream)
    h = None if residual is None else _new_like(x, x.dtype, stream)
    rstd = _new(x.shape[:-1], torch.float32, x, stream)
    rc = lib.dion_rmsnorm(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), _ptr(h), cols, y.data_ptr(), cols,
                          rstd.data_ptr(), rows, cols, code, wcode, eps, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, x, weight, residual)
    return y, (x if h is None else h), rstd


def rmsnorm_int8(x, weight, residual=None, eps=1e-6, stream=None):
    """The same norm written as 8-bit codes: returns (q, scale, h), y = q * scale.

    ``scale`` (fp32, one for each row) is the row's largest |y| over 127; a row
    that holds an infinity or a NaN has scale NaN."""
    dev, rows, cols, ldx, ldr, code, wcode = _norm_inputs(x, weight, residual)
    q = _new_like(x, torch.int8, stream)
    h = None if residual is None else _new_like(x, x.dtype, stream)
    scale = _new(x.shape[:-1], torch.float32, x, stream)
    rc = lib.dion_rmsnorm_int8(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), _ptr(h), cols, q.data_ptr(),
                               cols, scale.data_ptr(), rows, cols, code, wcode, eps, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, x, weight, residual)
    return q, scale, (x if h is None else h)


def rmsnorm_backward(dy, h, weight, rstd, dh=None, workspace=None, stream=None):
    """Gradients (dx, dweight) of ``rmsnorm`` from its ``h`` and ``rstd``.

    ``dh`` is the gradient that reaches h itself along the residual stream; dx
    is the gradient of x and of the residual alike."""
    dev = _device(h, "h")
    rows, cols, ldh = _matrix(h, "h")
    code = _code(h.dtype, "h")
    lddy = _same(dy, "dy", h, dev)
    lddh = 0 if dh is None else _same(dh, "dh", h, dev)
    _vector(weight, "weight", cols, (h.dtype, torch.float32), dev)
    _vector(rstd, "rstd", rows, _F32, dev)
    keep, ws, have = _workspace(lib.dion_rmsnorm_backward_workspace_size(rows, cols, code), h, workspace, stream)
    dx = _new_like(h, h.dtype, stream)
    dw = _new_like(weight, weight.dtype, stream)
    rc = lib.dion_rmsnorm_backward(dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(),
                                   _ptr(dh), lddh, dx.data_ptr(), cols, dw.data_ptr(), rows, cols, code,
                                   _CODE[weight.dtype], ws, have, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, dy, h, weight, rstd, dh, keep)
    return dx, dw


# ------------------------------------------------------------- 8-bit products
def int8_quantize(x, stream=None):
    """8-bit codes of the rows of x: returns (q, scale), x = q * scale up to rounding.
    (The weights of a product, once; activations that no norm wrote.)"""
    dev = _device(x, "x")
    rows, cols, ldx = _matrix(x, "x")
    code = _code(x.dtype, "x")
    q = _new_like(x, torch.int8, stream)
    scale = _new(x.shape[:-1], torch.float32, x, stream)
    rc = lib.dion_int8_quantize(x.data_ptr(), ldx, q.data_ptr(), cols, scale.data_ptr(), rows, cols, code,
                                _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, x)
    return q, scale


def int8_dequantize(q, scale, dtype=torch.bfloat16, stream=None):
    """The values that 8-bit codes with a scale for each row stand for."""
    dev = _device(q, "q")
    rows, cols, ldq = _matrix(q, "q")
    if q.dtype != torch.int8:
        _fail(f"q: expected torch.int8, got {q.dtype}")
    _vector(scale, "scale", rows, _F32, dev)
    code = _code(dtype, "dtype")
    y = _new_like(q, dtype, stream)
    rc = lib.dion_int8_dequantize(q.data_ptr(), ldq, scale.data_ptr(), y.data_ptr(), cols, rows, cols, code,
                                  _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, q, scale)
    return y


def int8_linear(a, a_scale, b, b_scale, bias=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """a (tokens x k) times b (channels x k) transposed, both int8, with a scale
    for each token and channel and an optional bias; the sum is exact."""
    dev = _device(a, "a")
    _beside(b, "b", dev)
    m, k, lda = _matrix(a, "a")
    n, kb, ldb = _matrix(b, "b")
    if a.dtype != torch.int8 or b.dtype != torch.int8:
        _fail(f"a and b must be int8, got {a.dtype} and {b.dtype}")
    if b.dim() != 2 or kb != k:
        _fail(f"b: shape {tuple(b.shape)}, expected (channels, {k})")
    _vector(a_scale, "a_scale", m, _F32, dev)
    _vector(b_scale, "b_scale", n, _F32, dev)
    code = _code(out_dtype, "out_dtype")
    if bias is not None:
        _vector(bias, "bias", n, _CODE, dev)
    pa, pb = a.data_ptr(), b.data_ptr()
    keep, ws, have = _scratch(lib.dion_int8_linear_workspace_size(pa, lda, pb, ldb, m, n, k), a, workspace, stream)
    out = _new((*a.shape[:-1], n), out_dtype, a, stream)
    rc = lib.dion_int8_linear(pa, lda, a_scale.data_ptr(), pb, ldb, b_scale.data_ptr(),
                              _ptr(bias), 0 if bias is None else _CODE[bias.dtype], out.data_ptr(), n, m, n, k, code,
                              ws, have, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, a, a_scale, b, b_scale, bias, keep)
    return out


# ---------------------------------------------------------------- distillation
def _dense(t, stream):
    """t itself, or a contiguous copy made on the stream that reads it"""
    if stream is None or t.is_contiguous():
        return t.contiguous()
    with torch.cuda.stream(stream):
        copy = t.contiguous()
    t.record_stream(stream)
    return copy


def _distill_inputs(logits, teacher, teacher_idx, stream):
    dev = _device(logits, "logits")
    rows, vocab, ldz = _matrix(logits, "logits")
    code = _code(logits.dtype, "logits")
    _beside(teacher, "teacher logits", dev)
    _beside(teacher_idx, "teacher indices", dev)
    shape = teacher.shape
    if len(shape) == 0 or shape != teacher_idx.shape or shape[:-1] != logits.shape[:-1]:
        _fail(f"teacher logits {tuple(shape)} and indices {tuple(teacher_idx.shape)} must be one row of "
              f"entries for each row of logits {tuple(logits.shape)}")
    tcode = _code(teacher.dtype, "teacher logits")
    if teacher_idx.dtype not in (torch.int64, torch.int32):
        _fail(f"teacher indices: unsupported dtype {teacher_idx.dtype}")
    return (dev, rows, vocab, ldz, code, _dense(teacher, stream), tcode, _dense(teacher_idx, stream),
            teacher_idx.element_size(), shape[-1])


def _gradient(logits, rows, vocab, out, stream, dev):
    """The gradient's tensor and row stride: new rows start at multiples of 16
    bytes, so that they are written in whole 16-byte pieces whatever the vocabulary."""
    if out is None:
        per = 16 // logits.element_size()
        wide = (vocab + per - 1) // per * per
        out = _new((*logits.shape[:-1], wide), logits.dtype, logits, stream)
        return (out if wide == vocab else out[..., :vocab]), (wide if rows > 1 else vocab)
    return out, _same(out, "out", logits, dev)


def distill_topk(logits, teacher, teacher_idx, temperature=1.0, workspace=None, stream=None):
    """Loss of each row against a teacher's top logits: returns (loss, stats).

    ``logits``: rows x vocab; ``teacher`` and ``teacher_idx`` (int64 or int32):
    rows x k.  loss = T^2 KL(p, q) with p the softmax of teacher / T over its k
    entries and q that of logits / T over the vocabulary; entries with an index
    outside the vocabulary or a logit of -inf are absent, and a row without any
    has loss and gradient 0.  ``stats`` is for ``distill_topk_backward``."""
    dev, rows, vocab, ldz, code, t, tcode, idx, ib, k = _distill_inputs(logits, teacher, teacher_idx, stream)
    keep, ws, have = _scratch(lib.dion_distill_topk_workspace_size(rows, vocab, k, code, 0), logits, workspace, stream)
    loss = _new(logits.shape[:-1], torch.float32, logits, stream)
    stats = _new((*logits.shape[:-1], 2), torch.float32, logits, stream)
    rc = lib.dion_distill_topk(logits.data_ptr(), ldz, t.data_ptr(), idx.data_ptr(), loss.data_ptr(), stats.data_ptr(),
                               rows, vocab, k, code, tcode, ib, temperature, ws, have, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, logits, t, idx, keep)
    return loss, stats


def distill_topk_backward(grad_loss, logits, stats, teacher, teacher_idx, temperature=1.0, out=None, stream=None):
    """Gradient of the logits from ``distill_topk``'s stats and the gradient of
    each row's loss (None: 1).  ``out`` may be the logits themselves."""
    dev, rows, vocab, ldz, code, t, tcode, idx, ib, k = _distill_inputs(logits, teacher, teacher_idx, stream)
    if grad_loss is not None:
        _vector(grad_loss, "grad_loss", rows, _F32, dev)
    _vector(stats, "stats", 2 * rows, _F32, dev)
    out, ldd = _gradient(logits, rows, vocab, out, stream, dev)
    rc = lib.dion_distill_topk_backward(_ptr(grad_loss), logits.data_ptr(), ldz, stats.data_ptr(), t.data_ptr(),
                                        idx.data_ptr(), out.data_ptr(), ldd, rows, vocab, k, code, tcode, ib,
                                        temperature, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, grad_loss, logits, stats, t, idx, out)
    return out


def distill_topk_step(logits, teacher, teacher_idx, grad_loss=None, temperature=1.0, out=None, workspace=None,
                      stream=None):
    """Loss and gradient in one call, for a ``grad_loss`` known ahead (such as
    one over the number of tokens; None: 1): returns (loss, dlogits).
    ``out`` may be the logits themselves."""
    dev, rows, vocab, ldz, code, t, tcode, idx, ib, k = _distill_inputs(logits, teacher, teacher_idx, stream)
    if grad_loss is not None:
        _vector(grad_loss, "grad_loss", rows, _F32, dev)
    keep, ws, have = _scratch(lib.dion_distill_topk_workspace_size(rows, vocab, k, code, 1), logits, workspace, stream)
    loss = _new(logits.shape[:-1], torch.float32, logits, stream)
    out, ldd = _gradient(logits, rows, vocab, out, stream, dev)
    rc = lib.dion_distill_topk_step(logits.data_ptr(), ldz, t.data_ptr(), idx.data_ptr(), _ptr(grad_loss),
                                    loss.data_ptr(), out.data_ptr(), ldd, rows, vocab, k, code, tcode, ib, temperature,
                                    ws, have, _handle(stream, dev))
    if rc:
        check(rc)
    _used(stream, logits, t, idx, grad_loss, out, keep)
    return loss, out


# ------------------------------------------------------------------- autograd
class _Gradient(torch.autograd.Function):
    """A gradient as a function of what it depends on, whose own derivative is refused."""

    @staticmethod
    def forward(ctx, compute, *tensors):
        return compute(*tensors)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("trying to differentiate twice: rms_norm and distill_loss have first derivatives only")


def _once(compute, *tensors):
    """compute(*tensors), the gradients of a backward pass.  Where a graph of that pass is asked for (create_graph),
    they carry one that raises: without it a second derivative would be missing silently."""
    return _Gradient.apply(compute, *tensors) if torch.is_grad_enabled() else compute(*tensors)


def _rows(t):
    """t, or a contiguous copy where it is no matrix of rows that the operators take (transposed, expanded)"""
    if not isinstance(t, torch.Tensor) or t.is_contiguous():
        return t
    try:
        _, cols, ld = _matrix(t, "")
    except DionError:
        return t.contiguous()
    return t if ld >= cols else t.contiguous()


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = rmsnorm(x, weight, residual, eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.residual = residual is not None
        ctx.set_materialize_grads(False)   # an output that nothing used sends None, not zeros to be read
        return (y, h) if ctx.residual else y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        if dy is None:
            return dh, None, dh, None
        dx, dw = _once(lambda dy, h, weight, dh: rmsnorm_backward(dy.contiguous(), h, weight, rstd,
                                                                  None if dh is None else dh.contiguous()),
                       dy, h, weight, dh)
        return dx, dw, (dx if ctx.residual else None), None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """``rmsnorm`` for automatic differentiation, once: returns y, or (y, h) with a residual.
    Tensors of any strides; what does not lie in rows is copied first."""
    return _RmsNorm.apply(_rows(x), _rows(weight), _rows(residual), eps)


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher, teacher_idx, temperature):
        loss, stats = distill_topk(logits, teacher, teacher_idx, temperature)
        ctx.save_for_backward(logits, stats, teacher, teacher_idx)
        ctx.temperature = temperature
        return loss

    @staticmethod
    def backward(ctx, grad):
        logits, stats, teacher, idx = ctx.saved_tensors
        dlogits = _once(lambda grad, logits: distill_topk_backward(grad.contiguous(), logits, stats, teacher, idx,
                                                                   ctx.temperature), grad, logits)
        return dlogits, None, None, None


def distill_loss(logits, teacher, teacher_idx, temperature=1.0):
    """``distill_topk`` for automatic differentiation, once: the loss of each row.
    The logits get a gradient, the teacher's do not.  Tensors of any strides, as
    for ``rms_norm``."""
    return _DistillLoss.apply(_rows(logits), teacher, teacher_idx, temperature)
