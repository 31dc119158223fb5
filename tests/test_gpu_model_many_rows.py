"""More rows than a grid has blocks (2^20, times the rows of a block): the kernels' loops over rows.  Every row's result is
that of the same row among few, bit for bit where the same kernel takes both."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layernorm_of_many_rows(dion, dtype):
    rows, cols = 17 * (1 << 20) + 5, 3   # 16 rows to a block
    x, w, b = randn(1, (1000, cols), dtype), randn(2, (cols,), dtype), randn(3, (cols,), dtype)
    many = x.repeat((rows + 999) // 1000, 1)[:rows].contiguous()
    y, _, mean, rstd = dion.layernorm(many, w, b)
    dx, dw, db = dion.layernorm_backward(many, many, w, mean, rstd)
    few = dion.layernorm(x, w, b)
    for got, want in ((y, few[0]), (mean, few[2]), (rstd, few[3]),
                      (dx, dion.layernorm_backward(x, x, w, few[2], few[3])[0])):
        assert torch.equal(got, want.repeat((rows + 999) // 1000, *[1] * (want.dim() - 1))[:rows])
    # sums over 1.8e7 rows: 1089 partial sums in turn to a thread, 1024 of them joined, each addition off by 2^-24 of its sum,
    # below 2^-13 of the magnitudes; then rounded to the weight's type
    v = (many.double() - mean.double()[:, None]) * rstd.double()[:, None]
    u = torch.finfo(dtype).eps / 2
    for got, terms in ((dw, many.double() * v), (db, many.double())):
        assert ((got.double() - terms.sum(0)).abs() <= u * terms.sum(0).abs() + 2.0 ** -13 * terms.abs().sum(0)).all()


def test_codes_of_many_rows(dion):
    rows = (1 << 25) + 77   # 16 rows to a block, two or four to a thread
    x = randn(1, (1000, 2), torch.bfloat16)
    many = x.repeat((rows + 999) // 1000, 1)[:rows].contiguous()
    q, s = dion.mxfp4_quantize(many)
    fq, fs = dion.mxfp4_quantize(x)
    assert torch.equal(q, fq.repeat((rows + 999) // 1000, 1)[:rows]) and torch.equal(s, fs.repeat((rows + 999) // 1000, 1)[:rows])
    back = dion.mxfp4_dequantize(q, s)
    assert torch.equal(back, dion.mxfp4_dequantize(fq, fs).repeat((rows + 999) // 1000, 1)[:rows])


@pytest.mark.parametrize("vocab,k", [(5, 3), (300, 20)])
def test_log_probabilities_of_many_rows(dion, vocab, k):
    rows = (1 << 20) + 1003   # a row to a block
    z = randn(1, (1000, vocab), torch.bfloat16)
    z[7] = -float("inf")
    z[8] = torch.finfo(torch.bfloat16).min
    z[9] = 1.0
    t = torch.arange(1000, device="cuda") % vocab
    t[5] = -1
    rep = lambda v: v.repeat((rows + 999) // 1000, *[1] * (v.dim() - 1))[:rows].contiguous()
    many, tokens = rep(z), rep(t)
    for got, want in zip(dion.top_logprobs(many, k, tokens), dion.top_logprobs(z, k, t)):
        assert torch.equal(got, rep(want))
    lp, ent, stats = dion.token_logprobs(many, tokens)
    few = dion.token_logprobs(z, t)
    for got, want in zip((lp, ent, stats), few):
        assert torch.equal(got, rep(want))
    one = torch.ones(1000, device="cuda")
    d = dion.token_logprobs_backward(rep(one), rep(one), many, stats, tokens)
    assert torch.equal(d, rep(dion.token_logprobs_backward(one, one, z, few[2], t)))


def test_products_of_many_rows(dion):
    """Tokens and channels up to the millions, on either side."""
    rows = (1 << 20) + 33
    (a, sa), (b, sb) = dion.mxfp4_quantize(randn(1, (1000, 64), torch.bfloat16)), dion.mxfp4_quantize(randn(2, (9, 64), torch.bfloat16))
    rep = lambda v: v.repeat((rows + 999) // 1000, 1)[:rows].contiguous()
    few = dion.mxfp4_dequantize(a, sa, torch.float32).double() @ dion.mxfp4_dequantize(b, sb, torch.float32).double().t().contiguous()
    mag = dion.mxfp4_dequantize(a, sa, torch.float32).double().abs() @ dion.mxfp4_dequantize(b, sb, torch.float32).double().abs().t().contiguous()
    for y in (dion.mxfp4_linear(rep(a), rep(sa), b, sb, out_dtype=torch.float32),
              dion.mxfp4_linear(b, sb, rep(a), rep(sa), out_dtype=torch.float32).t()):
        assert ((y.double() - rep(few)).abs() <= 81 * 2.0 ** -23 * rep(mag)).all()   # 64 terms, in fp32
