"""The C entry points of the training-step operators without a GPU: sizes and refusals, all before any launch.
Pointers are numbers that nothing dereferences."""
import ctypes

import pytest

import orthogonalized_optimizer_step_amd as dion  # noqa: F401
from orthogonalized_optimizer_step_amd import _lib

lib = _lib.lib
BF16, FP32, FP16 = 0, 1, 2
A, B, C, D, E, F, G, H = (0x10000000 * i for i in range(1, 9))   # far apart
INVAL, UNSUPPORTED, WORKSPACE = -1, -2, -3


def norm(x=A, ldx=64, r=B, ldr=64, w=C, h=D, ldh=64, y=E, ldy=64, stat=F, rows=4, cols=64, dt=BF16, wdt=BF16, eps=1e-6,
         int8=False):
    f = lib.dion_rmsnorm_int8 if int8 else lib.dion_rmsnorm
    return f(x, ldx, r, ldr, w, h, ldh, y, ldy, stat, rows, cols, dt, wdt, eps, None)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INVAL), (dict(w=None), INVAL), (dict(y=None), INVAL), (dict(stat=None), INVAL),
    (dict(rows=-1), INVAL), (dict(cols=0), INVAL), (dict(cols=65537, ldx=70000, ldr=70000, ldh=70000, ldy=70000), UNSUPPORTED),
    (dict(dt=3), INVAL), (dict(wdt=FP16), INVAL), (dict(eps=-1.0), INVAL), (dict(eps=float("nan")), INVAL),
    (dict(eps=float("inf")), INVAL), (dict(ldx=63), INVAL), (dict(ldh=10), INVAL), (dict(ldy=63), INVAL),
    (dict(x=A + 1), INVAL), (dict(y=A), INVAL), (dict(y=A + 2 * 64 * 3), INVAL), (dict(h=A + 2), INVAL),
    (dict(h=E), INVAL), (dict(stat=A), INVAL), (dict(stat=C), INVAL), (dict(y=C), INVAL), (dict(h=A, ldh=80), INVAL),
])
def test_norm_refusals(bad, code, int8):
    assert norm(int8=int8, **bad) == code
    assert lib.dion_last_error()


def test_no_rows_is_no_work():
    assert norm(rows=0, x=None, r=None, h=None, y=None, stat=None) == 0
    assert lib.dion_int8_quantize(None, 8, None, 8, None, 0, 8, BF16, None) == 0
    assert lib.dion_int8_dequantize(None, 8, None, None, 8, 0, 8, BF16, None) == 0
    assert lib.dion_int8_linear(None, 8, None, A, 8, B, None, 0, None, 8, 0, 8, 8, BF16, None, 0, None) == 0
    assert lib.dion_distill_topk(None, 8, None, None, None, None, 0, 8, 2, BF16, BF16, 8, 1.0, None, 0, None) == 0


def test_norm_backward_refusals():
    size = lib.dion_rmsnorm_backward_workspace_size

    def call(dy=A, h=B, w=C, rstd=D, dh=E, dx=F, dw=G, rows=100, cols=64, dt=BF16, wdt=BF16, ws=H, have=1 << 30):
        return lib.dion_rmsnorm_backward(dy, cols, h, cols, w, rstd, dh, cols, dx, cols, dw, rows, cols, dt, wdt, ws,
                                         have, None)

    need = size(100, 64, BF16)
    assert need > 0 and need % 256 == 0
    assert size(1 << 40, 64, BF16) < 1 << 24        # the partial sums do not grow with the rows
    assert size(-1, 64, BF16) == 0 and size(1, 0, BF16) == 0 and size(1, 65537, BF16) == 0 and size(1, 1, 9) == 0
    for bad, code in ((dict(dy=None), INVAL), (dict(rstd=None), INVAL), (dict(dw=None), INVAL), (dict(dx=B), INVAL),
                      (dict(dx=A + 2), INVAL), (dict(dw=A), INVAL), (dict(ws=None), WORKSPACE),
                      (dict(ws=H + 8), WORKSPACE), (dict(have=need - 1), WORKSPACE), (dict(ws=A, have=need), INVAL),
                      (dict(dt=7), INVAL), (dict(wdt=FP16), INVAL), (dict(rows=-3), INVAL)):
        assert call(**bad) == code, bad


def test_int8_linear_refusals_and_sizes():
    size = lib.dion_int8_linear_workspace_size

    def call(a=A, lda=64, sa=B, b=C, ldb=64, sb=D, bias=None, bdt=0, out=E, ldo=32, m=16, n=32, k=64, odt=BF16, ws=H,
             have=1 << 30):
        return lib.dion_int8_linear(a, lda, sa, b, ldb, sb, bias, bdt, out, ldo, m, n, k, odt, ws, have, None)

    assert size(A, 64, B, 64, 1, 64, 64) == 256                         # none
    assert size(A, 4096, B, 4096, 8192, 14336, 4096) == 256
    split = size(A, 14336, B, 14336, 24, 4096, 14336)
    assert split >= 2 * 24 * 4096 * 4                                   # sums of splits
    odd = size(A, 777, B, 777, 333, 1001, 777)
    assert odd >= (333 + 1001) * 784                                    # aligned copies of both
    assert 1001 * 784 > size(A + 1, 784, B, 784, 333, 1001, 784) >= 333 * 784   # of a alone
    assert size(A, 8, B, 8, -1, 1, 8) == 0 and size(A, 8, B, 8, 1, 1, 1 << 17) == 0
    for bad, code in ((dict(a=None), INVAL), (dict(sa=None), INVAL), (dict(sb=None), INVAL), (dict(out=None), INVAL),
                      (dict(lda=63), INVAL), (dict(ldo=31), INVAL), (dict(m=-1), INVAL), (dict(k=-1), INVAL),
                      (dict(k=1 << 17, lda=1 << 17, ldb=1 << 17), UNSUPPORTED), (dict(odt=5), INVAL),
                      (dict(bias=F, bdt=4), INVAL), (dict(out=A), INVAL), (dict(out=D), INVAL), (dict(out=E + 1), INVAL),
                      (dict(m=24, n=4096, k=14336, lda=14336, ldb=14336, ldo=4096, ws=None), WORKSPACE),
                      (dict(m=24, n=4096, k=14336, lda=14336, ldb=14336, ldo=4096, have=split - 1), WORKSPACE),
                      (dict(m=24, n=4096, k=14336, lda=14336, ldb=14336, ldo=4096, ws=H + 16), WORKSPACE),
                      (dict(m=24, n=4096, k=14336, lda=14336, ldb=14336, ldo=4096, ws=C), INVAL)):
        assert call(**bad) == code, bad


def test_distill_refusals_and_sizes():
    size = lib.dion_distill_topk_workspace_size

    def fwd(z=A, ldz=500, t=B, i=C, loss=D, stats=E, rows=4, vocab=500, k=8, dt=BF16, tdt=FP32, ib=8, temp=1.0, ws=None,
            have=0):
        return lib.dion_distill_topk(z, ldz, t, i, loss, stats, rows, vocab, k, dt, tdt, ib, temp, ws, have, None)

    def step(z=A, ldz=500, t=B, i=C, gl=F, loss=D, dz=G, ldd=500, rows=4, vocab=500, k=8, dt=BF16, tdt=FP32, ib=8,
             temp=1.0, ws=None, have=0):
        return lib.dion_distill_topk_step(z, ldz, t, i, gl, loss, dz, ldd, rows, vocab, k, dt, tdt, ib, temp, ws, have,
                                          None)

    def back(z=A, ldz=500, t=B, i=C, gl=F, stats=E, dz=G, ldd=500, rows=4, vocab=500, k=8, dt=BF16, tdt=FP32, ib=8,
             temp=1.0):
        return lib.dion_distill_topk_backward(gl, z, ldz, stats, t, i, dz, ldd, rows, vocab, k, dt, tdt, ib, temp, None)

    assert size(4, 500, 8, BF16, 1) == 256
    shared = size(4, 128000, 8, BF16, 1)
    assert shared > 256 and size(4, 128000, 8, BF16, 0) == 256 and size(4096, 128000, 8, BF16, 1) == 256
    assert size(-1, 5, 1, BF16, 1) == 0 and size(1, 0, 1, BF16, 1) == 0 and size(1, 5, 1025, BF16, 1) == 0
    common = ((dict(z=None), INVAL), (dict(t=None), INVAL), (dict(i=None), INVAL), (dict(rows=-1), INVAL),
              (dict(vocab=0), INVAL), (dict(k=-1), INVAL), (dict(k=1025), UNSUPPORTED), (dict(dt=3), INVAL),
              (dict(tdt=-1), INVAL), (dict(ib=2), INVAL), (dict(temp=0.0), INVAL), (dict(temp=-1.0), INVAL),
              (dict(temp=float("nan")), INVAL), (dict(temp=float("inf")), INVAL), (dict(ldz=499), INVAL),
              (dict(vocab=(1 << 30) + 1, ldz=1 << 31), UNSUPPORTED))
    for f in (fwd, step, back):
        for bad, code in common:
            assert f(**bad) == code, (f, bad)
    for bad in (dict(loss=None), dict(stats=None), dict(stats=E + 4), dict(loss=A), dict(stats=B), dict(loss=E)):
        assert fwd(**bad) == INVAL, bad
    for bad in (dict(loss=None), dict(dz=None), dict(dz=A + 2), dict(dz=A, ldd=600), dict(dz=C), dict(dz=F), dict(loss=G),
                dict(ldd=100)):
        assert step(**bad) == INVAL, bad
    for bad in (dict(stats=None), dict(stats=E + 4), dict(dz=E), dict(dz=A + 2), dict(dz=None)):
        assert back(**bad) == INVAL, bad
    big = dict(vocab=128000, ldz=128000, ldd=128000)
    assert step(**big) == WORKSPACE and step(ws=H, have=shared - 1, **big) == WORKSPACE
    assert step(ws=H + 4, have=shared, **big) == WORKSPACE and step(ws=A, have=shared, **big) == INVAL
