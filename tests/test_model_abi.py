"""The C entry points of the layer norm, the 4-bit operators and the log probabilities without a GPU: sizes and refusals,
all before any launch.  Pointers are numbers that nothing dereferences."""
import pytest

import orthogonalized_optimizer_step_amd as dion  # noqa: F401
from orthogonalized_optimizer_step_amd import _lib

lib = _lib.lib
BF16, FP32, FP16 = 0, 1, 2
A, B, C, D, E, F, G, H, I, J, K = (0x10000000 * i for i in range(1, 12))   # far apart
INVAL, UNSUPPORTED, WORKSPACE = -1, -2, -3


def norm(x=A, ldx=64, r=B, ldr=64, w=C, b=D, h=E, ldh=64, y=F, ldy=64, mean=G, rstd=H, rows=4, cols=64, dt=BF16, wdt=BF16,
         eps=1e-6):
    return lib.dion_layernorm(x, ldx, r, ldr, w, b, h, ldh, y, ldy, mean, rstd, rows, cols, dt, wdt, eps, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), INVAL), (dict(w=None), INVAL), (dict(y=None), INVAL), (dict(mean=None), INVAL), (dict(rstd=None), INVAL),
    (dict(rows=-1), INVAL), (dict(cols=0), INVAL),
    (dict(cols=65537, ldx=70000, ldr=70000, ldh=70000, ldy=70000), UNSUPPORTED), (dict(rows=(1 << 40) + 1), UNSUPPORTED),
    (dict(dt=3), INVAL), (dict(wdt=FP16), INVAL), (dict(eps=-1.0), INVAL), (dict(eps=float("nan")), INVAL),
    (dict(eps=float("inf")), INVAL), (dict(ldx=63), INVAL), (dict(ldh=10), INVAL), (dict(ldy=63), INVAL),
    (dict(x=A + 1), INVAL), (dict(b=D + 1), INVAL), (dict(y=A), INVAL), (dict(h=A + 2), INVAL), (dict(h=F), INVAL),
    (dict(mean=A), INVAL), (dict(mean=C), INVAL), (dict(rstd=D), INVAL), (dict(y=C), INVAL), (dict(y=D), INVAL),
    (dict(mean=H), INVAL), (dict(mean=F), INVAL), (dict(rstd=E), INVAL), (dict(h=A, ldh=80), INVAL), (dict(y=E), INVAL),
])
def test_layernorm_refusals(bad, code):
    assert norm(**bad) == code
    assert lib.dion_last_error()


def test_layernorm_backward_refusals():
    size = lib.dion_layernorm_backward_workspace_size

    def call(dy=A, h=B, w=C, mean=D, rstd=E, dh=F, dx=G, dw=H, db=I, rows=100, cols=64, dt=BF16, wdt=BF16, ws=J,
             have=1 << 30):
        return lib.dion_layernorm_backward(dy, cols, h, cols, w, mean, rstd, dh, cols, dx, cols, dw, db, rows, cols, dt,
                                           wdt, ws, have, None)

    need = size(100, 64, BF16)
    assert need > 0 and need % 256 == 0
    assert size(1 << 40, 64, BF16) < 1 << 24        # the partial sums do not grow with the rows
    assert size(-1, 64, BF16) == 0 and size(1, 0, BF16) == 0 and size(1, 65537, BF16) == 0 and size(1, 1, 9) == 0
    for bad, code in ((dict(dy=None), INVAL), (dict(mean=None), INVAL), (dict(rstd=None), INVAL), (dict(dw=None), INVAL),
                      (dict(dx=None), INVAL), (dict(dx=B), INVAL), (dict(dx=A + 2), INVAL), (dict(dw=A), INVAL),
                      (dict(db=H), INVAL), (dict(db=F), INVAL), (dict(db=I + 1), INVAL), (dict(ws=None), WORKSPACE),
                      (dict(ws=J + 8), WORKSPACE), (dict(have=need - 1), WORKSPACE), (dict(ws=A, have=need), INVAL),
                      (dict(ws=I, have=need), INVAL), (dict(dt=7), INVAL), (dict(wdt=FP16), INVAL), (dict(rows=-3), INVAL)):
        assert call(**bad) == code, bad


def codes(read, x=A, ldx=100, q=B, ldq=50, s=C, lds=4, rows=4, cols=100, dt=BF16):
    if read:
        return lib.dion_mxfp4_dequantize(q, ldq, s, lds, x, ldx, rows, cols, dt, None)
    return lib.dion_mxfp4_quantize(x, ldx, q, ldq, s, lds, rows, cols, dt, None)


@pytest.mark.parametrize("read", [False, True])
def test_mxfp4_codes_refusals(read):
    for bad, code in ((dict(x=None), INVAL), (dict(q=None), INVAL), (dict(s=None), INVAL), (dict(ldx=99), INVAL),
                      (dict(ldq=49), INVAL), (dict(lds=3), INVAL), (dict(rows=-1), INVAL), (dict(cols=0), INVAL),
                      (dict(dt=4), INVAL), (dict(x=A + 1), INVAL), (dict(q=A), INVAL), (dict(s=A), INVAL),
                      (dict(rows=(1 << 40) + 1), UNSUPPORTED), (dict(cols=-5), INVAL),
                      (dict(cols=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 30, lds=1 << 26), UNSUPPORTED)):
        assert codes(read, **bad) == code, bad
    assert read or codes(read, q=C) == INVAL


def test_mxfp4_linear_refusals_and_sizes():
    size = lambda a, lda, sa, ldsa, b, ldb, sb, ldsb, m, n, k: lib.dion_mxfp4_linear_workspace_size(
        a, lda, sa, ldsa, b, ldb, sb, ldsb, m, n, k)

    def call(a=A, lda=32, sa=B, ldsa=2, b=C, ldb=32, sb=D, ldsb=2, bias=None, bdt=0, out=E, ldo=32, m=16, n=32, k=64,
             odt=BF16, ws=H, have=1 << 30):
        return lib.dion_mxfp4_linear(a, lda, sa, ldsa, b, ldb, sb, ldsb, bias, bdt, out, ldo, m, n, k, odt, ws, have, None)

    assert size(A, 32, B, 2, C, 32, D, 2, 1, 64, 64) == 256                              # none
    assert size(A, 2048, B, 128, C, 2048, D, 128, 8192, 14336, 4096) == 256
    split = size(A, 7168, B, 448, C, 7168, D, 448, 24, 4096, 14336)
    assert split >= 2 * 24 * 4096 * 4                                                    # sums of splits
    odd = size(A, 389, B, 25, C, 389, D, 25, 333, 1001, 778)
    assert odd >= (333 + 1001) * (400 + 32)                                              # aligned copies of all four
    assert 1001 * 16 <= size(A, 256, B, 16, C, 256, D + 1, 16, 333, 1001, 512) < 1001 * 256   # of one's scales
    assert size(A, 8, B, 1, C, 8, D, 1, -1, 1, 8) == 0 and size(A, 8, B, 1, C, 8, D, 1, 1, 1, 7) == 0
    assert size(A, 8, B, 1, C, 8, D, 1, 1, 1, (1 << 22) + 2) == 0
    big = dict(m=24, n=4096, k=14336, lda=7168, ldb=7168, ldsa=448, ldsb=448, ldo=4096)
    for bad, code in ((dict(a=None), INVAL), (dict(sa=None), INVAL), (dict(b=None), INVAL), (dict(sb=None), INVAL),
                      (dict(out=None), INVAL), (dict(lda=31), INVAL), (dict(ldsa=1), INVAL), (dict(ldo=31), INVAL),
                      (dict(m=-1), INVAL), (dict(k=-2), INVAL), (dict(k=63), INVAL),
                      (dict(k=(1 << 22) + 2, lda=1 << 22, ldb=1 << 22, ldsa=1 << 20, ldsb=1 << 20), UNSUPPORTED),
                      (dict(m=(1 << 22) + 1), UNSUPPORTED), (dict(odt=5), INVAL), (dict(bias=F, bdt=4), INVAL),
                      (dict(out=A), INVAL), (dict(out=D), INVAL), (dict(out=E + 1), INVAL),
                      (dict(ws=None, **big), WORKSPACE), (dict(have=split - 1, **big), WORKSPACE),
                      (dict(ws=H + 16, **big), WORKSPACE), (dict(ws=C, **big), INVAL)):
        assert call(**bad) == code, bad


# k in splits whose sums fit 256 bytes, and copies of a few unaligned rows
@pytest.mark.parametrize("m,n,k,off", [(1, 1, 14336, 0), (2, 16, 14336, 0), (17, 1, 512, 1), (17, 1, 32, 0)])
def test_little_scratch_is_asked_for_and_checked(m, n, k, off):
    args = (A + off, k // 2, B, k // 32, C, k // 2, D, k // 32)
    need = lib.dion_mxfp4_linear_workspace_size(*args, m, n, k)
    assert need > 256

    def call(ws, have):
        return lib.dion_mxfp4_linear(*args, None, 0, E, n, m, n, k, BF16, ws, have, None)

    assert call(None, 0) == WORKSPACE and call(None, need) == WORKSPACE
    assert call(H, 0) == WORKSPACE and call(H, need - 1) == WORKSPACE and call(H + 16, need) == WORKSPACE
    assert call(A, need) == INVAL   # on top of an operand


def test_logprobs_refusals():
    size = lib.dion_token_logprobs_workspace_size

    def fwd(z=A, ldz=500, t=B, lp=C, ent=D, stats=E, top=F, index=G, rows=4, vocab=500, k=8, dt=BF16, tb=8, temp=1.0,
            ws=None, have=0):
        return lib.dion_token_logprobs(z, ldz, t, lp, ent, stats, top, index, rows, vocab, k, dt, tb, temp, ws, have, None)

    def back(z=A, ldz=500, t=B, gl=C, ge=D, stats=E, dz=F, ldd=500, rows=4, vocab=500, dt=BF16, tb=8, temp=1.0):
        return lib.dion_token_logprobs_backward(gl, ge, z, ldz, stats, t, dz, ldd, rows, vocab, dt, tb, temp, None)

    common = ((dict(z=None), INVAL), (dict(rows=-1), INVAL), (dict(vocab=0), INVAL), (dict(dt=3), INVAL),
              (dict(tb=2), INVAL), (dict(temp=0.0), INVAL), (dict(temp=-1.0), INVAL), (dict(temp=float("nan")), INVAL),
              (dict(temp=float("inf")), INVAL), (dict(temp=1e-39), INVAL), (dict(ldz=499), INVAL), (dict(z=A + 1), INVAL), (dict(t=B + 4), INVAL),
              (dict(vocab=(1 << 30) + 1, ldz=1 << 31), UNSUPPORTED), (dict(rows=(1 << 40) + 1), UNSUPPORTED))
    for f in (fwd, back):
        for bad, code in common:
            assert f(**bad) == code, (f, bad)
    for bad, code in ((dict(lp=None), INVAL), (dict(ent=None), INVAL), (dict(top=None), INVAL), (dict(index=None), INVAL),
                      (dict(k=-1), INVAL), (dict(k=1025), UNSUPPORTED),
                      (dict(vocab=(1 << 19) + 1, ldz=1 << 20), UNSUPPORTED), (dict(stats=E + 4), INVAL),
                      (dict(lp=A), INVAL), (dict(ent=B), INVAL), (dict(ent=C), INVAL), (dict(top=G), INVAL),
                      (dict(index=E), INVAL), (dict(stats=A), INVAL), (dict(index=G + 4), INVAL)):
        assert fwd(**bad) == code, bad
    assert size(4, 500, 8, BF16) == 256 and size(4096, 128256, 64, BF16) == 256 and size(0, 128256, 64, BF16) == 256
    for bad in ((-1, 5, 1, BF16), (1, 0, 1, BF16), (1, 5, 1025, BF16), (1, 5, -1, BF16), (1, (1 << 19) + 1, 1, BF16), (1, 5, 1, 3)):
        assert size(*bad) == 0
    for rows, vocab, k in ((1, 128256, 20), (1, 128256, 0), (4, 100000, 32), (1, 128256, 1)):
        need, big = size(rows, vocab, k, BF16), dict(rows=rows, vocab=vocab, ldz=vocab, k=k)
        assert need > 256
        assert fwd(**big) == WORKSPACE and fwd(ws=H, have=need - 1, **big) == WORKSPACE
        assert fwd(ws=H + 8, have=need, **big) == WORKSPACE
        for on in (A, B, C, D, E) + ((F, G) if k else ()):
            assert fwd(ws=on, have=need, **big) == INVAL
    for bad in (dict(stats=None), dict(stats=E + 8), dict(dz=None), dict(dz=A + 2), dict(dz=A, ldd=600), dict(dz=B),
                dict(dz=C), dict(dz=D), dict(dz=E), dict(ldd=100), dict(gl=C + 2)):
        assert back(**bad) == INVAL, bad


def test_no_rows_is_no_work():
    assert norm(rows=0, x=None, r=None, h=None, y=None, mean=None, rstd=None) == 0
    assert lib.dion_mxfp4_quantize(None, 8, None, 4, None, 1, 0, 8, BF16, None) == 0
    assert lib.dion_mxfp4_dequantize(None, 4, None, 1, None, 8, 0, 8, BF16, None) == 0
    assert lib.dion_mxfp4_linear(None, 4, None, 1, A, 4, B, 1, None, 0, None, 8, 0, 8, 8, BF16, None, 0, None) == 0
    assert lib.dion_token_logprobs(None, 8, None, None, None, None, None, None, 0, 8, 2, BF16, 8, 1.0, None, 0, None) == 0
    assert lib.dion_token_logprobs_backward(None, None, None, 8, None, None, None, 8, 0, 8, BF16, 8, 1.0, None) == 0
