"""The layer norm's gradient without those of its weight and bias: dx is that of the whole gradient bit for bit, from the
entry points and under automatic differentiation, in place, on a stream and in a graph."""
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


SHAPES = [(0, 64), (1, 1), (9, 63), (5, 128), (33, 257), (130, 768), (1000, 1001), (40, 4096), (7, 8200), (3, 16384), (5, 20001)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                         (torch.float32, torch.float32)])
@pytest.mark.parametrize("stream", [False, True])
def test_dx_alone(dion, rows, cols, dtype, wtype, stream):
    x, r, dy, dh = (randn(i, (rows, cols), dtype) for i in range(4))
    w = randn(5, (cols,), wtype)
    _, h, mean, rstd = dion.layernorm(x, w, residual=r)
    side = torch.cuda.Stream() if stream else None
    for along in (dh, None):
        want = dion.layernorm_backward(dy, h, w, mean, rstd, dh=along)[0]
        dx, dw, db = dion.layernorm_backward(dy, h, w, mean, rstd, dh=along, only_dx=True, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(dx, want) and dw is None and db is None


@pytest.mark.parametrize("cols", [100, 4096, 20001])
def test_dx_alone_over_its_inputs(dion, cols):
    from orthogonalized_optimizer_step_amd._lib import lib
    x, dy, dh = (randn(i, (9, cols), torch.bfloat16) for i in range(3))
    w = randn(5, (cols,), torch.bfloat16)
    _, h, mean, rstd = dion.layernorm(x, w)
    want = dion.layernorm_backward(dy, h, w, mean, rstd, dh=dh)[0]
    for into in (0, 1):
        g = [dy.clone(), dh.clone()]
        assert lib.dion_layernorm_backward_dx(g[0].data_ptr(), cols, h.data_ptr(), cols, w.data_ptr(), mean.data_ptr(),
                                              rstd.data_ptr(), g[1].data_ptr(), cols, g[into].data_ptr(), cols, 9, cols, 0, 0,
                                              None) == 0
        torch.cuda.synchronize()
        assert torch.equal(g[into], want) and torch.equal(g[1 - into], (dy, dh)[1 - into])


@pytest.mark.parametrize("w,b", [(True, False), (False, True), (False, False)])
def test_frozen_weights_under_automatic_differentiation(dion, w, b):
    x, r, gy, gh = (randn(i, (40, 300), torch.bfloat16) for i in range(4))
    weight, bias = randn(5, (300,), torch.bfloat16), randn(6, (300,), torch.bfloat16)
    leaves = [t.clone().requires_grad_() for t in (x, r, weight, bias)]
    torch.autograd.backward(dion.layer_norm(leaves[0], leaves[2], leaves[3], leaves[1]), (gy, gh))
    some = [t.clone().requires_grad_(on) for t, on in ((x, True), (r, True), (weight, w), (bias, b))]
    torch.autograd.backward(dion.layer_norm(some[0], some[2], some[3], some[1]), (gy, gh))
    for a, c, on in zip(some, leaves, (True, True, w, b)):
        assert torch.equal(a.grad, c.grad) if on else a.grad is None


def test_dx_alone_in_a_graph(dion):
    x, dy = randn(1, (300, 768), torch.bfloat16), randn(2, (300, 768), torch.bfloat16)
    w = randn(3, (768,), torch.bfloat16)
    _, h, mean, rstd = dion.layernorm(x, w)
    want = dion.layernorm_backward(dy, h, w, mean, rstd)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx = dion.layernorm_backward(dy, h, w, mean, rstd, only_dx=True)[0]
    for _ in range(3):
        dx.zero_()
        eager = dion.layernorm_backward(dy, h, w, mean, rstd, only_dx=True)[0]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want) and torch.equal(eager, want)
