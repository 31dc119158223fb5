"""The oracle of the layer norm, the 4-bit codes and the log probabilities against torch's own operators, automatic
differentiation and differences, in float64 on the CPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import model_oracle as O  # noqa: E402


def test_layernorm_and_its_gradient_against_autograd():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(5, 37, generator=g, dtype=torch.float64) + 2).requires_grad_()
    w, b = (torch.randn(37, generator=g, dtype=torch.float64).requires_grad_() for _ in range(2))
    dy = torch.randn(5, 37, generator=g, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (37,), w, b, 1e-3)
    y.backward(dy)
    got, mean, rstd = O.layernorm(x.detach().numpy(), w.detach().numpy(), b.detach().numpy(), 1e-3)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db = O.layernorm_backward(dy.numpy(), x.detach().numpy(), w.detach().numpy(), mean, rstd)
    for a, t in ((dx, x), (dw, w), (db, b)):
        np.testing.assert_allclose(a, t.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_mx_codes_are_the_nearest_with_the_least_scale():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((40, 100)) * 10.0 ** rng.integers(-30, 30, (40, 1))
    code, scale = O.mx_codes(x)
    v = O.mx_values(O.mx_pack(code), scale, 100)
    step = 2.0 ** (np.repeat(scale.astype(np.float64) - 127, 32, 1)[:, :100])
    a = np.abs(x) / step
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0))
    assert (np.abs(x - v) / step <= half).all() and a.max() < 7 and (a.reshape(40, -1).max(1) >= 3.5).all()
    # ties, the smallest scale, and blocks that hold no number
    t = np.zeros((4, 32))
    t[0, :8] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    t[1, :2] = 7, -7
    t[2, 0] = 2.0 ** -140
    t[3, 0] = np.nan
    code, scale = O.mx_codes(t)
    assert list(code[0, :8]) == [6, 0, 2, 2, 4, 4, 6, 6] and scale[0, 0] == 127
    assert scale[1, 0] == 128 and list(code[1, :2]) == [6, 14] and scale[2, 0] == 0 and scale[3, 0] == 255


def test_logprobs_and_gradient_against_autograd():
    g = torch.Generator().manual_seed(3)
    z = (torch.randn(6, 50, generator=g, dtype=torch.float64) * 3)
    z[2, 10:] = -np.inf
    z = z.requires_grad_()
    tokens = np.array([3, 0, 5, -1, 50, 49])
    T = 0.7
    logq = torch.log_softmax(z / T, 1)
    q = logq.exp()
    ent = -torch.where(q > 0, q * torch.where(q > 0, logq, torch.zeros(())), torch.zeros(())).sum(1)
    lp = torch.stack([logq[i, t] if 0 <= t < 50 else torch.zeros((), dtype=torch.float64) for i, t in enumerate(tokens)])
    gl, ge = torch.randn(6, generator=g, dtype=torch.float64), torch.randn(6, generator=g, dtype=torch.float64)
    (lp @ gl + ent @ ge).backward()
    a, e, _, _ = O.logprobs(z.detach().numpy(), tokens, T)
    np.testing.assert_allclose(a, lp.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(e, ent.detach().numpy(), rtol=1e-12)
    d = O.logprobs_backward(gl.numpy(), ge.numpy(), z.detach().numpy(), tokens, T)
    np.testing.assert_allclose(d, np.nan_to_num(z.grad.numpy()), rtol=1e-9, atol=1e-12)


def test_top_orders_equal_logits_by_index():
    z = np.array([[1.0, 3, 3, -np.inf, 2], [-np.inf] * 5, [0.0, -0.0, 0.0, -1, -np.inf]])
    assert O.top(z, 4).tolist() == [[1, 2, 4, 0], [-1] * 4, [0, 1, 2, 3]]
