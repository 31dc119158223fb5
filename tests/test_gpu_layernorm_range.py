"""Layer norms at the ends of the fp32 range and of rows that hold no number: the statistics that are returned, and what the
gradient makes of them.  What is compared is exact."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


def randn(seed, shape, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


COLS = [100, 500, 1001, 4096, 40000]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e25, 1e28, 1e32])
def test_rows_whose_squares_overflow(dion, cols, dtype, size):
    """Squares of 1e20 and more are no fp32 numbers, sums of 40000 elements of 1e32 are: rstd is 0 and y the bias, whatever
    the first mean was off by (1e25 and its square: the correction's own square overflows too)."""
    x = randn(1, (6, cols), dtype) + 1
    clean = x.clone()
    x[1] *= size
    x[4] *= -size
    w, b = randn(2, (cols,), dtype), randn(3, (cols,), dtype)
    y, h, mean, rstd = dion.layernorm(x, w, b)
    assert not rstd[[1, 4]].any() and torch.isfinite(mean).all()
    assert torch.equal(y[1], b) and torch.equal(y[4], b)
    some = [0, 2, 3, 5]
    cy, ch, cmean, crstd = dion.layernorm(clean, w, b)
    assert torch.equal(y[some], cy[some]) and torch.equal(rstd[some], crstd[some]) and torch.equal(mean[some], cmean[some])
    # its gradient, at rstd 0: none by way of the norm, what comes along the residual stream, and the bias's
    dy, dh = randn(4, (6, cols), dtype), randn(5, (6, cols), dtype)
    dx, dw, db = dion.layernorm_backward(dy, h, w, mean, rstd, dh=dh)
    assert torch.equal(dx[[1, 4]], dh[[1, 4]]) and torch.isfinite(dw).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_statistics_of_rows_that_hold_no_number(dion, cols, dtype, bad):
    """mean, rstd, y and dx of such a row are NaN, the others' are what they are without it."""
    x = randn(1, (5, cols), dtype)
    x[3, cols // 2] = bad
    w, b, dy = randn(2, (cols,), dtype), randn(3, (cols,), dtype), randn(4, (5, cols), dtype)
    y, h, mean, rstd = dion.layernorm(x, w, b)
    assert torch.isnan(y[3]).all() and torch.isnan(rstd[3]) and not torch.isfinite(mean[3])
    dx, _, _ = dion.layernorm_backward(dy, h, w, mean, rstd)
    assert torch.isnan(dx[3]).all()
    some = [0, 1, 2, 4]
    cy, ch, cmean, crstd = dion.layernorm(x[some], w, b)
    assert torch.equal(y[some], cy) and torch.equal(mean[some], cmean) and torch.equal(rstd[some], crstd)
    assert torch.equal(dx[some], dion.layernorm_backward(dy[some], ch, w, cmean, crstd)[0])
