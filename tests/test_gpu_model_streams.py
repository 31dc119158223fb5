"""The ``stream`` argument of the layer norm, the 4-bit operators and the log probabilities, for tensors that the current
stream is still making, and inside a captured graph.  Everything is equal bit for bit."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


def randn(seed, shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def calls(dion):
    """name, inputs, call"""
    x, r, w, b = randn(1, (64, 320)), randn(2, (64, 320)), randn(3, (320,)), randn(4, (320,))
    _, h, mean, rstd = dion.layernorm(x, w, b, residual=r)
    q, s = dion.mxfp4_quantize(x)
    hq, hs = dion.mxfp4_quantize(randn(5, (700, 320)))
    z, t = randn(6, (64, 3001)), torch.randint(3001, (64, 2), device="cuda")
    stats = dion.token_logprobs(z, t[:, 0])[2]
    one = torch.ones(64, device="cuda")
    return [
        ("layernorm", (x, w, b, r), lambda s, x, w, b, r: dion.layernorm(x, w, b, residual=r, stream=s)),
        ("layernorm_backward", (r, h, w, mean, rstd, x),
         lambda s, dy, h, w, m, r, dh: dion.layernorm_backward(dy, h, w, m, r, dh=dh, stream=s)),
        ("mxfp4_quantize", (x,), lambda s, x: dion.mxfp4_quantize(x, stream=s)),
        ("mxfp4_dequantize", (q, s), lambda s, q, e: (dion.mxfp4_dequantize(q, e, stream=s),)),
        ("mxfp4_linear", (q, s, hq, hs), lambda s, *a: (dion.mxfp4_linear(*a, stream=s),)),
        ("token_logprobs", (z, t), lambda s, z, t: dion.token_logprobs(z, t[:, 1], stream=s)),
        ("top_logprobs", (z, t), lambda s, z, t: dion.top_logprobs(z, 9, t[:, 1], stream=s)),
        ("token_logprobs_backward", (one, one, z, stats, t),
         lambda s, gl, ge, z, st, t: (dion.token_logprobs_backward(gl, ge, z, st, t[:, 0], stream=s),)),
    ]


def test_tensors_that_the_current_stream_is_still_making(dion):
    side = torch.cuda.Stream()
    busy = randn(7, (4096, 4096), torch.float32)
    for name, inputs, call in calls(dion):
        want = call(None, *inputs)
        late = [torch.full_like(t, 77) for t in inputs]   # what lies there before
        torch.cuda.synchronize()
        for _ in range(20):   # a few ms and more on the current stream
            busy = busy @ busy * 1e-3
        for t, v in zip(late, inputs):
            t.copy_(v)
        got = call(side, *late)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("forked", [False, True])
def test_a_given_stream_in_a_captured_graph(dion, forked):
    """The stream joins the graph by the call or was made part of it before, and goes back to it by the caller."""
    side = torch.cuda.Stream()
    for name, inputs, call in calls(dion):
        want = [t.clone() for t in call(None, *inputs)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if forked:
                side.wait_stream(torch.cuda.current_stream())
            out = call(side, *inputs)
            torch.cuda.current_stream().wait_stream(side)
        for _ in range(3):
            for t in out:
                t.zero_()
            eager = call(None, *inputs)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), name
            assert all(torch.equal(a, b) for a, b in zip(eager, want)), name
