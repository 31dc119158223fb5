"""The float64 oracle of the training-step operators: its gradients against central differences of its own forward
passes, its values against hand-worked small cases (CPU)."""
import numpy as np
import pytest

from oracle import train_oracle as O


def difference(f, x, at, step):
    up, down = x.copy(), x.copy()
    up[at] += step
    down[at] -= step
    return (f(up) - f(down)) / (2 * step)


@pytest.mark.parametrize("rows,cols,eps", [(1, 1, 1e-6), (3, 7, 1e-5), (4, 33, 0.1)])
def test_rmsnorm_gradient_against_differences(rows, cols, eps):
    rng = np.random.default_rng(rows * 100 + cols)
    h, dy, dh = (rng.standard_normal((rows, cols)) for _ in range(3))
    w = 1 + 0.3 * rng.standard_normal(cols)
    dx, dw = O.rmsnorm_backward(dy, h, w, eps, dh)
    for at in np.ndindex(rows, cols):
        d = difference(lambda v: (O.rmsnorm(v, w, eps)[0] * dy).sum() + (v * dh).sum(), h, at, 1e-5)
        assert abs(d - dx[at]) <= 1e-7 * max(1.0, abs(dx[at]))
    for j in range(cols):
        d = difference(lambda v: (O.rmsnorm(h, v, eps)[0] * dy).sum(), w, j, 1e-5)
        assert abs(d - dw[j]) <= 1e-7 * max(1.0, abs(dw[j]))


@pytest.mark.parametrize("temp", [0.5, 1.0, 3.0])
def test_distill_gradient_against_differences(temp):
    rng = np.random.default_rng(4)
    z, t = 2 * rng.standard_normal((4, 9)), 2 * rng.standard_normal((4, 5))
    idx = np.array([[0, 8, 3, 2, 5], [1, 1, 4, -1, 99], [7, 6, 5, 4, 3], [-1, -1, -1, -1, 9]])
    t[2, 1] = -np.inf
    loss, dz, live = O.distill(z, t, idx, temp)
    assert list(live) == [True, True, True, False]
    assert loss[3] == 0 and not dz[3].any()
    for at in np.ndindex(4, 9):
        d = difference(lambda v: O.distill(v, t, idx, temp)[0].sum(), z, at, 1e-5)
        assert abs(d - dz[at]) <= 1e-7


def test_distill_small_case_by_hand():
    # one teacher entry: p = 1, loss = T^2 * (lse(z / T) - z_i / T)
    z = np.array([[1.0, 2.0, 3.0]])
    loss, dz, _ = O.distill(z, np.array([[5.0]]), np.array([[1]]), 2.0)
    lse = np.log(np.exp(0.5) + np.exp(1.0) + np.exp(1.5))
    assert abs(loss[0] - 4 * (lse - 1.0)) < 1e-12
    q = np.exp(z[0] / 2 - lse)
    assert np.allclose(dz[0], 2 * (q - np.array([0, 1, 0])), atol=1e-12)
    # the teacher's own distribution as the student: no loss, no gradient
    t = np.array([[0.3, -0.7, 1.1]])
    loss, dz, _ = O.distill(t, t, np.array([[0, 1, 2]]), 1.0)
    assert abs(loss[0]) < 1e-12 and np.abs(dz).max() < 1e-12


def test_int8_linear_by_hand():
    y = O.int8_linear([[127, -128]], [0.5], [[-128, 127], [1, 2]], [2.0, 1.0], [1.0, -1.0])
    assert y.tolist() == [[-32511.0, -65.5]]
