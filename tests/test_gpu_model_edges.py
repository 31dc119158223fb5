"""Layer norm, microscaled 4-bit operators and log probabilities on the GPU: what they must leave alone, given and shared
workspaces, outputs over inputs, captured graphs and streams side by side, and alternatives at the edges of their lists.

What is compared here is equal bit for bit, or between whole numbers: there are no tolerances.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import model_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu

GUARD = 64   # elements before and behind an output


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


@pytest.fixture(scope="module")
def lib():
    from orthogonalized_optimizer_step_amd._lib import lib
    return lib


CODE = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


def randn(seed, shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


class Held:
    """rows x cols of an output inside a larger allocation of a byte pattern, its rows `gap` elements further apart than
    they are long and its first at element GUARD + `off`."""

    def __init__(self, rows, cols, dtype, gap=0, off=0):
        self.rows, self.cols, self.ld, self.at = rows, cols, cols + gap, GUARD + off
        size = torch.empty(0, dtype=dtype).element_size()
        self.bytes = torch.full(((2 * GUARD + off + rows * self.ld) * size,), 0xa5, dtype=torch.uint8, device="cuda")
        self.all = self.bytes.view(dtype)

    @property
    def ptr(self):
        return self.all[self.at:].data_ptr()

    @property
    def value(self):
        return self.all[self.at:self.at + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols]

    def beside_is_untouched(self):
        rest = torch.ones(self.all.shape, dtype=torch.bool, device="cuda")
        rest[self.at:self.at + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = False
        return bool((self.bytes.view(rest.numel(), -1)[rest] == 0xa5).all())


def ok(*held):
    torch.cuda.synchronize()
    for i, h in enumerate(held):
        assert h.beside_is_untouched(), i


# ------------------------------------------------- nothing is written beside an output
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols,gap,off", [(1, 1, 0, 1), (5, 7, 3, 1), (9, 63, 1, 0), (130, 130, 0, 3), (3, 1001, 5, 1),
                                               (2, 8193, 1, 1), (2, 20001, 0, 1), (70, 520, 8, 0)])
def test_layernorm_writes_its_outputs_only(dion, lib, dtype, rows, cols, gap, off):
    x, r, dy, dh = (randn(i, (rows, cols), dtype) for i in range(4))
    w, b = randn(5, (cols,), dtype), randn(6, (cols,), dtype)
    y, h, dx = (Held(rows, cols, dtype, gap, off) for _ in range(3))
    mean, rstd, dw, db = Held(1, rows, torch.float32), Held(1, rows, torch.float32), Held(1, cols, dtype), Held(1, cols, dtype)
    code = CODE[dtype]
    assert lib.dion_layernorm(x.data_ptr(), cols, r.data_ptr(), cols, w.data_ptr(), b.data_ptr(), h.ptr, h.ld, y.ptr, y.ld,
                              mean.ptr, rstd.ptr, rows, cols, code, code, 1e-5, None) == 0
    need = lib.dion_layernorm_backward_workspace_size(rows, cols, code)
    ws = Held(1, need, torch.uint8, 0, 192)   # at a multiple of 256 bytes
    assert lib.dion_layernorm_backward(dy.data_ptr(), cols, h.ptr, h.ld, w.data_ptr(), mean.ptr, rstd.ptr, dh.data_ptr(),
                                       cols, dx.ptr, dx.ld, dw.ptr, db.ptr, rows, cols, code, code, ws.ptr, need, None) == 0
    ok(y, h, mean, rstd, dx, dw, db, ws)
    wy, wh, wm, wr = dion.layernorm(x, w, b, residual=r)
    for got, want in ((y, wy), (h, wh), (mean, wm[None]), (rstd, wr[None])):
        assert torch.equal(got.value, want)
    for got, want in zip((dx, dw, db), dion.layernorm_backward(dy, wh, w, wm, wr, dh=dh)):
        assert torch.equal(got.value, want if want.dim() == 2 else want[None])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,gap,off", [(1, 1, 0, 1), (3, 5, 1, 3), (7, 33, 0, 1), (5, 96, 3, 2), (2, 4100, 1, 1),
                                               (40, 1024, 0, 0)])
def test_mxfp4_codes_write_their_outputs_only(dion, lib, dtype, rows, cols, gap, off):
    x = randn(1, (rows, cols), dtype)
    q, s = Held(rows, (cols + 1) // 2, torch.uint8, gap, off), Held(rows, (cols + 31) // 32, torch.uint8, gap, off)
    y = Held(rows, cols, dtype, gap, off)
    assert lib.dion_mxfp4_quantize(x.data_ptr(), cols, q.ptr, q.ld, s.ptr, s.ld, rows, cols, CODE[dtype], None) == 0
    assert lib.dion_mxfp4_dequantize(q.ptr, q.ld, s.ptr, s.ld, y.ptr, y.ld, rows, cols, CODE[dtype], None) == 0
    ok(q, s, y)
    wq, ws = dion.mxfp4_quantize(x)
    assert torch.equal(q.value, wq) and torch.equal(s.value, ws)
    assert torch.equal(y.value, dion.mxfp4_dequantize(wq, ws, dtype, cols=cols))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 64), (1, 37, 14336), (16, 14000, 512), (17, 33, 70), (130, 129, 1026), (300, 1001, 512),
                                   (24, 70, 8192), (1024, 2600, 512)])
@pytest.mark.parametrize("gap,off", [(0, 0), (3, 1)])
def test_mxfp4_linear_writes_its_output_only(dion, lib, out, m, n, k, gap, off):
    a, sa = dion.mxfp4_quantize(randn(1, (m, k)))
    b, sb = dion.mxfp4_quantize(randn(2, (n, k)))
    bias = randn(3, (n,))
    args = (a.data_ptr(), k // 2, sa.data_ptr(), sa.shape[1], b.data_ptr(), k // 2, sb.data_ptr(), sb.shape[1])
    need = lib.dion_mxfp4_linear_workspace_size(*args, m, n, k)
    ws, y = Held(1, need, torch.uint8, 0, 192), Held(m, n, out, gap, off)
    assert lib.dion_mxfp4_linear(*args, bias.data_ptr(), 0, y.ptr, y.ld, m, n, k, CODE[out], ws.ptr, need, None) == 0
    ok(ws, y)
    assert torch.equal(y.value, dion.mxfp4_linear(a, sa, b, sb, bias, out))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 3), (3, 501, 5), (300, 257, 8), (2, 70001, 300), (2, 100001, 20), (1, 128256, 0),
                                          (40, 9001, 0)])
def test_logprobs_write_their_outputs_only(dion, lib, dtype, rows, vocab, k):
    z = randn(1, (rows, vocab), dtype)
    t = torch.arange(rows, device="cuda") % vocab
    lp, ent, stats = Held(1, rows, torch.float32), Held(1, rows, torch.float32), Held(rows, 4, torch.float32)
    top, index, dz = Held(rows, k, torch.float32), Held(rows, k, torch.int64), Held(rows, vocab, dtype, 3, 1)
    need = lib.dion_token_logprobs_workspace_size(rows, vocab, k, CODE[dtype])
    ws = Held(1, need, torch.uint8, 0, 192)
    assert lib.dion_token_logprobs(z.data_ptr(), vocab, t.data_ptr(), lp.ptr, ent.ptr, stats.ptr, top.ptr, index.ptr, rows,
                                   vocab, k, CODE[dtype], 8, 1.0, ws.ptr, need, None) == 0
    assert lib.dion_token_logprobs_backward(lp.ptr, ent.ptr, z.data_ptr(), vocab, stats.ptr, t.data_ptr(), dz.ptr, dz.ld,
                                            rows, vocab, CODE[dtype], 8, 1.0, None) == 0
    ok(lp, ent, stats, top, index, dz, ws)
    wtop, windex, wlp, went = dion.top_logprobs(z, k, t)
    assert torch.equal(lp.value[0], wlp) and torch.equal(ent.value[0], went)
    assert torch.equal(top.value, wtop) and torch.equal(index.value, windex)
    want = dion.token_logprobs_backward(wlp, went, z, stats.value.contiguous(), t)
    assert torch.equal(dz.value, want)


# ------------------------------------------------- outputs over inputs
@pytest.mark.parametrize("cols", [100, 1001, 4096, 20001])
def test_layernorm_over_its_inputs(lib, dion, cols):
    x, r, dy, dh = (randn(i, (9, cols)) for i in range(4))
    w, b = randn(5, (cols,)), randn(6, (cols,))
    y, h, mean, rstd = dion.layernorm(x, w, b, residual=r)
    want = dion.layernorm_backward(dy, h, w, mean, rstd, dh=dh)
    for into in (0, 1):
        c = [x.clone(), r.clone()]
        y2, m2, s2 = torch.empty_like(x), torch.empty_like(mean), torch.empty_like(rstd)
        assert lib.dion_layernorm(c[0].data_ptr(), cols, c[1].data_ptr(), cols, w.data_ptr(), b.data_ptr(),
                                  c[into].data_ptr(), cols, y2.data_ptr(), cols, m2.data_ptr(), s2.data_ptr(), 9, cols, 0, 0,
                                  1e-5, None) == 0
        assert torch.equal(c[into], h) and torch.equal(y2, y) and torch.equal(m2, mean) and torch.equal(s2, rstd)
        g = [dy.clone(), dh.clone()]
        dw, db = torch.empty_like(w), torch.empty_like(w)
        need = lib.dion_layernorm_backward_workspace_size(9, cols, 0)
        ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        assert lib.dion_layernorm_backward(g[0].data_ptr(), cols, h.data_ptr(), cols, w.data_ptr(), mean.data_ptr(),
                                           rstd.data_ptr(), g[1].data_ptr(), cols, g[into].data_ptr(), cols, dw.data_ptr(),
                                           db.data_ptr(), 9, cols, 0, 0, ws.data_ptr() + -ws.data_ptr() % 256, need,
                                           None) == 0
        for got, ref in zip((g[into], dw, db), want):
            assert torch.equal(got, ref)


# ------------------------------------------------- workspaces
def products(dion):
    """Products whose k is split, and log probabilities whose rows are shared out, which join parts in a workspace; and a
    product that uses none (the second)."""
    b, sb = dion.mxfp4_quantize(randn(1, (256, 8192)))
    long, sl = dion.mxfp4_quantize(randn(6, (48, 28672)))
    return [(lambda ws, a=a: dion.mxfp4_linear(*a, b, sb, out_dtype=torch.float32, workspace=ws))
            for a in (dion.mxfp4_quantize(randn(2, (24, 8192))), dion.mxfp4_quantize(randn(3, (3, 8192))))] + \
           [lambda ws: dion.mxfp4_linear(long[:3], sl[:3], long, sl, workspace=ws)] + \
           [(lambda ws, z=z: torch.cat([v.double().flatten() for v in dion.top_logprobs(z, 20, workspace=ws)[:2]]))
            for z in (randn(4, (2, 128256)), randn(5, (9, 60000), torch.float32))]


def test_one_workspace_for_calls_in_turn(dion):
    calls = products(dion)
    want = [f(None) for f in calls]
    ws = torch.full((1 << 24,), 0xff, dtype=torch.uint8, device="cuda")   # whatever it holds
    for _ in range(2):
        for f, w in zip(calls, want):
            assert torch.equal(f(ws), w)
    for f in calls[:1] + calls[2:]:
        with pytest.raises(dion.DionError):
            f(ws[:600])
        with pytest.raises(dion.DionError):
            f(ws[::2])
        with pytest.raises(dion.DionError):
            f(torch.zeros(1 << 24, dtype=torch.uint8))


def test_two_graphs_beside_each_other(dion):
    """Captured with workspaces of their own, replayed in turn, then at once on two streams, between eager calls."""
    calls = products(dion)
    want = [f(None) for f in calls]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [f(None) for f in calls]
        graphs.append(g)
        outs.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        for out in outs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for i in (0, 1, 0):
            if turn < 2:
                graphs[i].replay()
            elif i == 0 or turn == 3:
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        eager = [f(None) for f in calls]
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            if turn == 2 and i == 1:
                continue
            for o, w in zip(out, want):
                assert torch.equal(o, w), (turn, i)
        for o, w in zip(eager, want):
            assert torch.equal(o, w), turn


def test_two_streams_at_once(dion):
    calls = products(dion)
    want = [f(None) for f in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([f(None) for f in calls])
    torch.cuda.synchronize()
    for out in got:
        for o, w in zip(out, want):
            assert torch.equal(o, w)


# ------------------------------------------------- alternatives at the edges of their lists
@pytest.mark.parametrize("rows", [1, 70, 300])
@pytest.mark.parametrize("vocab", [255, 2000, 4096, 32768, 32769, 65537])
@pytest.mark.parametrize("k", [128, 129, 255, 256, 257, 700])
def test_many_alternatives(dion, rows, vocab, k):
    """Rows whose largest lie apart, side by side in few groups, and with ties across the last place."""
    z = randn(rows + vocab + k, (rows, vocab))
    z[0, 3:3 + min(vocab - 3, 2 * k)] += 16                         # side by side
    if rows > 2:
        z[1] = z[1].round()                                         # many equal ones
        z[2] = torch.arange(vocab, device="cuda").remainder(97).to(z.dtype)
    index = dion.top_logprobs(z, k)[1]
    some = [0, 1, 2, rows - 1] if rows > 2 else [0]
    assert np.array_equal(index[some].cpu().numpy(), O.top(z[some].double().cpu().numpy(), k))


@pytest.mark.parametrize("temp", [1.1754944e-38, 1e-20, 1e20, 3e38])
def test_extreme_temperatures(dion, temp):
    """So cold that all of it is on the largest, so hot that all logits count alike: both to the last digits of fp32."""
    z = torch.tensor([[1.0, 3.0, -2.0, 3.0, 2.0], [-1.0, -8.0, -1.5, -9.0, -7.0]], device="cuda")
    t = torch.tensor([1, 0], device="cuda")
    lp, ent, stats = dion.token_logprobs(z, t, temperature=temp)
    dz = dion.token_logprobs_backward(torch.ones(2, device="cuda"), torch.ones(2, device="cuda"), z, stats, t, temperature=temp)
    ref = torch.tensor([2.0, 1.0], device="cuda").log() if temp < 1 else torch.full((2,), 5.0, device="cuda").log()
    assert torch.allclose(ent, ref, rtol=0, atol=2.0 ** -21) and torch.allclose(lp, -ref, rtol=0, atol=2.0 ** -21)
    assert torch.isfinite(dz).all()


def test_phases_are_recorded(dion):
    x, w = randn(1, (40, 64)), randn(2, (64,))
    dion.profile_enable(True)
    try:
        y, h, mean, rstd = dion.layernorm(x, w)
        dion.layernorm_backward(y, h, w, mean, rstd)
        q, s = dion.mxfp4_quantize(x)
        dion.mxfp4_dequantize(q, s)
        z = dion.mxfp4_linear(q, s, q, s)
        t = torch.zeros(40, dtype=torch.int64, device="cuda")
        _, _, stats = dion.token_logprobs(z, t)
        dion.token_logprobs_backward(mean, None, z, stats, t)
        torch.cuda.synchronize()
        names = [r[0] for r in dion.profile_records()]
    finally:
        dion.profile_enable(False)
    assert names == ["layernorm", "layernorm_backward", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_linear",
                     "token_logprobs", "token_logprobs_backward"]
