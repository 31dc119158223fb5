"""Which gradients of a layer norm automatic differentiation asks the library for, and the refusals of the entry point that
writes dx alone; without a GPU."""
import pytest

torch = pytest.importorskip("torch")

import orthogonalized_optimizer_step_amd.model_ops as M  # noqa: E402
from orthogonalized_optimizer_step_amd import _lib  # noqa: E402


@pytest.mark.parametrize("w,b", [(True, True), (True, False), (False, True), (False, False), (True, None), (False, None)])
@pytest.mark.parametrize("twice", [False, True])
def test_sums_are_formed_only_for_what_is_trained(monkeypatch, w, b, twice):
    asked = []

    def forward(x, weight, bias, residual, eps):
        h = x + residual
        return h * weight, h, h[:, 0], h[:, 0]

    def backward(dy, h, weight, mean, rstd, dh=None, bias=True, only_dx=False):
        asked.append((bias, only_dx))
        return dy * weight, None if only_dx else torch.ones_like(weight), torch.zeros_like(weight) if bias else None

    monkeypatch.setattr(M, "layernorm", forward)
    monkeypatch.setattr(M, "layernorm_backward", backward)
    x, r = (torch.randn(3, 5).requires_grad_() for _ in range(2))
    weight = torch.randn(5).requires_grad_(w)
    bias = None if b is None else torch.randn(5).requires_grad_(b)
    leaves = [t for t in (x, r, weight, bias) if t is not None and t.requires_grad]
    y, _ = M.layer_norm(x, weight, bias, r)
    grads = torch.autograd.grad(y.sum(), leaves, create_graph=twice)
    assert asked == [(bool(b), not (w or b))]
    assert torch.equal(grads[0], weight.expand(3, 5)) and torch.equal(grads[1], grads[0])
    assert all(torch.equal(g, torch.full((5,), v)) for g, v in zip(grads[2:], ([1.0] if w else []) + ([0.0] if b else [])))
    if twice:
        with pytest.raises(RuntimeError, match="differentiate twice"):
            grads[0].sum().backward()


A, B, C, D, E, F, G = (0x10000000 * i for i in range(1, 8))   # far apart
INVAL, UNSUPPORTED = -1, -2


def dx_alone(dy=A, h=B, w=C, mean=D, rstd=E, dh=F, dx=G, ld=64, rows=100, cols=64, dt=0, wdt=0):
    return _lib.lib.dion_layernorm_backward_dx(dy, ld, h, ld, w, mean, rstd, dh, ld, dx, ld, rows, cols, dt, wdt, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dy=None), INVAL), (dict(h=None), INVAL), (dict(w=None), INVAL), (dict(mean=None), INVAL),
    (dict(rstd=None), INVAL), (dict(dx=None), INVAL), (dict(dx=B), INVAL), (dict(dx=A + 2), INVAL), (dict(dx=C), INVAL),
    (dict(dx=D), INVAL), (dict(dx=E), INVAL), (dict(dx=F + 4), INVAL), (dict(dy=A + 1), INVAL), (dict(ld=63), INVAL),
    (dict(rows=-1), INVAL), (dict(cols=0), INVAL), (dict(cols=65537, ld=70000), UNSUPPORTED),
    (dict(rows=(1 << 40) + 1), UNSUPPORTED), (dict(dt=5), INVAL), (dict(wdt=2), INVAL)])
def test_refusals_of_dx_alone(bad, code):
    assert dx_alone(**bad) == code
    assert _lib.lib.dion_last_error()


def test_no_rows_is_no_work():
    assert dx_alone(rows=0, dy=None, h=None, mean=None, rstd=None, dh=None, dx=None) == 0
