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


def _gpu(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{what} must be a tensor on the GPU")
    if t.get_device() != torch.cuda.current_device():
        _fail(f"{what} is on another device than the current one")


def _matrix(t, what):
    """rows, cols and row stride of a tensor whose leading dimensions flatten into rows"""
    _gpu(t, what)
    if t.dim() != 2:
        if t.dim() == 0:
            _fail(f"{what} must have at least one dimension")
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(t.numel() // max(1, t.shape[-1]), t.shape[-1])
        except RuntimeError:
            _fail(f"{what}: the leading dimensions do not flatten into equally spaced rows")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1 and rows > 0:
        _fail(f"{what}: the elements of a row must be contiguous")
    return rows, cols, (t.stride(0) if rows > 1 else cols)


def _same(t, what, shape, dtype):
    if t.shape != shape:
        _fail(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        _fail(f"{what}: expected {dtype}, got {t.dtype}")
    return _matrix(t, what)[2]


def _vector(t, what, n, dtypes):
    _gpu(t, what)
    if t.numel() != n or (n > 1 and not t.is_contiguous()):
        _fail(f"{what} must be contiguous with {n} entries")
    if t.dtype not in dtypes:
        _fail(f"{what}: unsupported dtype {t.dtype}")
    return t


class _Stream:
    """The stream of a call: its handle, allocations that belong to it, and the tensors it uses."""

    def __init__(self, stream):
        self.stream = stream
        self.handle = (torch.cuda.current_stream() if stream is None else stream).cuda_stream

    def empty(self, shape, dtype, like):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=like.device)
        with torch.cuda.stream(self.stream):
            out = torch.empty(shape, dtype=dtype, device=like.device)
        out.record_stream(torch.cuda.current_stream())
        return out

    def workspace(self, nbytes, like, given):
        """address and length of the caller's workspace, or of a new one (kept alive by the returned tensor)"""
        if nbytes == 0:
            raise DionError(-1, lib.dion_last_error().decode())
        if given is None:
            given = self.empty(nbytes + 256, torch.uint8, like)
        at = given.data_ptr()
        off = -at % 256
        have = given.numel() * given.element_size() - off
        if have < nbytes:
            raise DionError(-3, f"workspace too small: need {nbytes} bytes")
        return given, at + off, have

    def used(self, *tensors):
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ RMS norm
def _norm_inputs(x, weight, residual):
    rows, cols, ldx = _matrix(x, "x")
    code = _code(x.dtype, "x")
    ldr = 0 if residual is None else _same(residual, "residual", x.shape, x.dtype)
    _vector(weight, "weight", cols, (x.dtype, torch.float32))
    return rows, cols, ldx, ldr, code, _CODE[weight.dtype]


def rmsnorm(x, weight, residual=None, eps=1e-6, stream=None):
    """RMS norm of the rows of ``x + residual``: returns (y, h, rstd).

    ``h`` is the sum in x's type, the residual stream carried on (x itself
    without a residual); ``rstd`` (fp32, one for each row) and ``h`` are what
    ``rmsnorm_backward`` needs.  ``weight``: x's type or fp32."""
    rows, cols, ldx, ldr, code, wcode = _norm_inputs(x, weight, residual)
    s = _Stream(stream)
    y = s.empty(x.shape, x.dtype, x)
    h = None if residual is None else s.empty(x.shape, x.dtype, x)
    rstd = s.empty(x.shape[:-1], torch.float32, x)
    check(lib.dion_rmsnorm(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), _ptr(h), cols, y.data_ptr(),
                           cols, rstd.data_ptr(), rows, cols, code, wcode, eps, s.handle))
    s.used(x, weight, residual)
    return y, (x if h is None else h), rstd


def rmsnorm_int8(x, weight, residual=None, eps=1e-6, stream=None):
    """The same norm written as 8-bit codes: returns (q, scale, h), y = q * scale.

    ``scale`` (fp32, one for each row) is the row's largest |y| over 127; a row
    that holds an infinity or a NaN has scale NaN."""
    rows, cols, ldx, ldr, code, wcode = _norm_inputs(x, weight, residual)
    s = _Stream(stream)
    q = s.empty(x.shape, torch.int8, x)
    h = None if residual is None else s.empty(x.shape, x.dtype, x)
    scale = s.empty(x.shape[:-1], torch.float32, x)
    check(lib.dion_rmsnorm_int8(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), _ptr(h), cols,
                                q.data_ptr(), cols, scale.data_ptr(), rows, cols, code, wcode, eps, s.handle))
    s.used(x, weight, residual)
    return q, scale, (x if h is None else h)


def rmsnorm_backward(dy, h, weight, rstd, dh=None, workspace=None, stream=None):
    """Gradients (dx, dweight) of ``rmsnorm`` from its ``h`` and ``rstd``.

    ``dh`` is the gradient that reaches h itself along the residual stream; dx
    is the gradient of x and of the residual alike."""
    rows, cols, ldh = _matrix(h, "h")
    code = _code(h.dtype, "h")
    lddy = _same(dy, "dy", h.shape, h.dtype)
    lddh = 0 if dh is None else _same(dh, "dh", h.shape, h.dtype)
    _vector(weight, "weight", cols, (h.dtype, torch.float32))
    _vector(rstd, "rstd", rows, (torch.float32,))
    s = _Stream(stream)
    keep, ws, have = s.workspace(lib.dion_rmsnorm_backward_workspace_size(rows, cols, code), h, workspace)
    dx = s.empty(h.shape, h.dtype, h)
    dw = s.empty(weight.shape, weight.dtype, h)
    check(lib.dion_rmsnorm_backward(dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(),
                                    _ptr(dh), lddh, dx.data_ptr(), cols, dw.data_ptr(), rows, cols, code,
                                    _CODE[weight.dtype], ws, have, s.handle))
    s.used(dy, h, weight, rstd, dh, keep)
    return dx, dw


# ------------------------------------------------------------- 8-bit products
def int8_quantize(x, stream=None):
    """8-bit codes of the rows of x: returns (q, scale), x = q * scale up to rounding.
    (The weights of a product, once; activations that no norm wrote.)"""
    rows, cols, ldx = _matrix(x, "x")
    code = _code(x.dtype, "x")
    s = _Stream(stream)
    q = s.empty(x.shape, torch.int8, x)
    scale = s.empty(x.shape[:-1], torch.float32, x)
    check(lib.dion_int8_quantize(x.data_ptr(), ldx, q.data_ptr(), cols, scale.data_ptr(), rows, cols, code, s.handle))
    s.used(x)
    return q, scale


def int8_dequantize(q, scale, dtype=torch.bfloat16, stream=None):
    """The values that 8-bit codes with a scale for each row stand for."""
    rows, cols, ldq = _matrix(q, "q")
    if q.dtype != torch.int8:
        _fail(f"q: expected torch.int8, got {q.dtype}")
    _vector(scale, "scale", rows, (torch.float32,))
    code = _code(dtype, "dtype")
    s = _Stream(stream)
    y = s.empty(q.shape, dtype, q)
    check(lib.dion_int8_dequantize(q.data_ptr(), ldq, scale.data_ptr(), y.data_ptr(), cols, rows, cols, code,
                                   s.handle))
    s.used(q, scale)
    return y


def int8_linear(a, a_scale, b, b_scale, bias=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """a (tokens x k) times b (channels x k) transposed, both int8, with a scale
    for each token and channel and an optional bias; the sum is exact."""
    m, k, lda = _matrix(a, "a")
    n, kb, ldb = _matrix(b, "b")
    if a.dtype != torch.int8 or b.dtype != torch.int8:
        _fail(f"a and b must be int8, got {a.dtype} and {b.dtype}")
    if b.dim() != 2 or kb != k:
        _fail(f"b: shape {tuple(b.shape)}, expected (channels, {k})")
    _vector(a_scale, "a_scale", m, (torch.float32,))
    _vector(b_scale, "b_scale", n, (torch.float32,))
    code = _code(out_dtype, "out_dtype")
    if bias is not None:
        _vector(bias, "bias", n, _CODE)
    s = _Stream(stream)
    keep, ws, have = s.workspace(lib.dion_int8_linear_workspace_size(m, n, k), a, workspace)
    out = s.empty((*a.shape[:-1], n), out_dtype, a)
    check(lib.dion_int8_linear(a.data_ptr(), lda, a_scale.data_ptr(), b.data_ptr(), ldb, b_scale.data_ptr(),
                               _ptr(bias), 0 if bias is None else _CODE[bias.dtype], out.data_ptr(), n, m, n, k, code,
                               ws, have, s.handle))
    s.used(a, a_scale, b, b_scale, bias, keep)
    return out


# ---------------------------------------------------------------- distillation
def _distill_inputs(logits, teacher, teacher_idx):
    rows, vocab, ldz = _matrix(logits, "logits")
    code = _code(logits.dtype, "logits")
    if teacher.dim() == 0 or teacher.shape != teacher_idx.shape or teacher.shape[:-1] != logits.shape[:-1]:
        _fail(f"teacher logits {tuple(teacher.shape)} and indices {tuple(teacher_idx.shape)} must be one row of "
              f"entries for each row of logits {tuple(logits.shape)}")
    _gpu(teacher, "teacher logits")
    _gpu(teacher_idx, "teacher indices")
    tcode = _code(teacher.dtype, "teacher logits")
    if teacher_idx.dtype not in (torch.int64, torch.int32):
        _fail(f"teacher indices: unsupported dtype {teacher_idx.dtype}")
    return (rows, vocab, ldz, code, teacher.contiguous(), tcode, teacher_idx.contiguous(),
            teacher_idx.element_size(), teacher.shape[-1])


def _gradient(s, logits, rows, vocab, out):
    """The gradient's tensor and row stride: new rows start at multiples of 16
    bytes, so that they are written in whole 16-byte pieces whatever the vocabulary."""
    if out is None:
        per = 16 // logits.element_size()
        wide = (vocab + per - 1) // per * per
        out = s.empty((*logits.shape[:-1], wide), logits.dtype, logits)[..., :vocab]
        return out, (wide if rows > 1 else vocab)
    return out, _same(out, "out", logits.shape, logits.dtype)


def distill_topk(logits, teacher, teacher_idx, temperature=1.0, workspace=None, stream=None):
    """Loss of each row against a teacher's top logits: returns (loss, stats).

    ``logits``: rows x vocab; ``teacher`` and ``teacher_idx`` (int64 or int32):
    rows x k.  loss = T^2 KL(p, q) with p the softmax of teacher / T over its k
    entries and q that of logits / T over the vocabulary; entries with an index
    outside the vocabulary or a logit of -inf are absent, and a row without any
    has loss and gradient 0.  ``stats`` is for ``distill_topk_backward``."""
    rows, vocab, ldz, code, t, tcode, idx, ib, k = _distill_inputs(logits, teacher, teacher_idx)
    s = _Stream(stream)
    keep, ws, have = s.workspace(lib.dion_distill_topk_workspace_size(rows, vocab), logits, workspace)
    loss = s.empty(logits.shape[:-1], torch.float32, logits)
    stats = s.empty((*logits.shape[:-1], 2), torch.float32, logits)
    check(lib.dion_distill_topk(logits.data_ptr(), ldz, t.data_ptr(), idx.data_ptr(), loss.data_ptr(),
                                stats.data_ptr(), rows, vocab, k, code, tcode, ib, temperature, ws, have, s.handle))
    s.used(logits, t, idx, keep)
    return loss, stats


def distill_topk_backward(grad_loss, logits, stats, teacher, teacher_idx, temperature=1.0, out=None, stream=None):
    """Gradient of the logits from ``distill_topk``'s stats and the gradient of
    each row's loss (None: 1).  ``out`` may be the logits themselves."""
    rows, vocab, ldz, code, t, tcode, idx, ib, k = _distill_inputs(logits, teacher, teacher_idx)
    if grad_loss is not None:
        _vector(grad_loss, "grad_loss", rows, (torch.float32,))
    _vector(stats, "stats", 2 * rows, (torch.float32,))
    s = _Stream(stream)
    out, ldd = _gradient(s, logits, rows, vocab, out)
    check(lib.dion_distill_topk_backward(_ptr(grad_loss), logits.data_ptr(), ldz, stats.data_ptr(), t.data_ptr(),
                                         idx.data_ptr(), out.data_ptr(), ldd, rows, vocab, k, code, tcode, ib,
                                         temperature, s.handle))
    s.used(grad_loss, logits, stats, t, idx, out)
    return out


def distill_topk_step(logits, teacher, teacher_idx, grad_loss=None, temperature=1.0, out=None, workspace=None,
                      stream=None):
    """Loss and gradient in one call, for a ``grad_loss`` known ahead (such as
    one over the number of tokens; None: 1): returns (loss, dlogits).
    ``out`` may be the logits themselves."""
    rows, vocab, ldz, code, t, tcode, idx, ib, k = _distill_inputs(logits, teacher, teacher_idx)
    if grad_loss is not None:
        _vector(grad_loss, "grad_loss", rows, (torch.float32,))
    s = _Stream(stream)
    keep, ws, have = s.workspace(lib.dion_distill_topk_workspace_size(rows, vocab), logits, workspace)
    loss = s.empty(logits.shape[:-1], torch.float32, logits)
    out, ldd = _gradient(s, logits, rows, vocab, out)
    check(lib.dion_distill_topk_step(logits.data_ptr(), ldz, t.data_ptr(), idx.data_ptr(), _ptr(grad_loss),
                                     loss.data_ptr(), out.data_ptr(), ldd, rows, vocab, k, code, tcode, ib,
                                     temperature, ws, have, s.handle))
    s.used(logits, t, idx, grad_loss, out, keep)
    return loss, out


# ------------------------------------------------------------------- autograd
class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = rmsnorm(x, weight, residual, eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.residual = residual is not None
        return (y, h) if ctx.residual else y

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        dx, dw = rmsnorm_backward(dy.contiguous(), h, weight, rstd, None if dh is None else dh.contiguous())
        return dx, dw, (dx if ctx.residual else None), None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """``rmsnorm`` for automatic differentiation: returns y, or (y, h) with a residual."""
    return _RmsNorm.apply(x, weight, residual, eps)


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
        return (distill_topk_backward(grad.contiguous(), logits, stats, teacher, idx, ctx.temperature), None, None,
                None)


def distill_loss(logits, teacher, teacher_idx, temperature=1.0):
    """``distill_topk`` for automatic differentiation: the loss of each row."""
    return _DistillLoss.apply(logits, teacher, teacher_idx, temperature)
