"""Layer norm, microscaled 4-bit operators and log probabilities on the GPU against the float64 oracle.

Tolerances.  u is the largest relative rounding error of the output's type (bf16 2^-8, fp16 2^-11, fp32 2^-24).  An fp32
sum of n terms in which no partial sum runs over more than 512 terms and a tree of 16 is off by at most 528 * 2^-24 <
2^-14 of the sum of magnitudes; rounding errors are that large only if all of them point one way.  ACC = 2^-15 allows
half of it.
  layer norm y     u |y| + ACC (2 |d rstd w| + |w|) + 2^-22 (|d rstd w| + |b|), d = s - mean (the mean is off by ACC of the
                   mean |d|, at most 1 / rstd); rstd 2 ACC; mean ACC mean|d| + 2^-23 |mean|
             dx    u |dx| + ACC rstd (|g| + mean|g| + |v| mean|g v|), v the normalised row
             dw    u |dw| + ACC sum |dy v|      db   u |db| + ACC sum |dy|
  4-bit codes and values: equal bit for bit
  product    u |out| + (k / 64 + 80) 2^-23 sum |a b| + 2^-23 (|product| + |bias|): one addition after another over k in
             steps of 64, up to 80 inside a step and where waves and splits meet, each off by 2^-23 of the magnitudes
  logprob    ACC + 2^-21 D, D = |u_t| + |log s| + entropy + 4 (u = (z - max) / T: two roundings of it in each exponential)
  entropy    (ACC + 2^-20 D) (1 + entropy), D without a token's u
  dlogits    u |dz| + (q (ACC + 2^-20 D_j) (|gl| + |ge| (1 + D_j)) + 2^-22 |gl| at the token) / T
fp16 results below its normal range round to multiples of 2^-24: 2^-25 is added.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import model_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ACC = 2.0 ** -15
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


def n64(t):
    return t.detach().double().cpu().numpy()


def strided(t, pad, off):
    """The same values in rows further apart, starting `off` elements into each."""
    if not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan") if t.is_floating_point() else 77, device=t.device)
    wide = wide.to(t.dtype)
    view = wide[:, off:off + t.shape[1]]
    view.copy_(t)
    return view


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(seed, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def within(got, ref, tol, what):
    got = n64(got) if isinstance(got, torch.Tensor) else got
    with np.errstate(all="ignore"):
        bad = ~((np.abs(got - ref) <= tol) | (got == ref))
        assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))))


# ---------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (3, 2), (2, 7), (5, 63), (4, 64), (17, 65), (130, 128), (9, 257), (65, 768), (33, 1001),
               (1, 4096), (3, 4097), (2, 8192), (5, 8200), (2, 16384), (2, 20001), (1, 65536), (700, 100)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype,wtype,residual,bias,pad", [
    ("bf16", "bf16", True, True, 0), ("fp16", "fp32", False, True, 3), ("fp32", "fp32", True, False, 5),
    ("bf16", "fp32", True, True, 16), ("fp16", "fp16", True, False, 0), ("fp32", "fp32", False, True, 0)])
def test_layernorm_forward_backward(dion, rows, cols, dtype, wtype, residual, bias, pad):
    dt, wd, eps = DT[dtype], DT[wtype], 1e-5
    x = strided(randn(1, (rows, cols), dt) + 0.5, pad, pad // 2)
    r = strided(randn(2, (rows, cols), dt, 3.0), pad, pad // 3) if residual else None
    w = (1 + 0.3 * randn(3, (cols,), torch.float32)).to(wd)
    b = randn(4, (cols,), wd) if bias else None
    s = x.float() + r.float() if residual else x.float()
    y, h, mean, rstd = dion.layernorm(x, w, b, residual=r, eps=eps)
    assert torch.equal(h, s.to(dt))
    S, W, B = n64(s), n64(w), None if b is None else n64(b)
    ref, mref, rref = O.layernorm(S, W, B, eps)
    d = S - mref[:, None]
    within(mean, mref, ACC * np.abs(d).mean(1) + 2.0 ** -23 * np.abs(mref) + 1e-37, "mean")
    within(rstd, rref, 2 * ACC * rref, "rstd")
    uw = np.abs(d * rref[:, None] * W)
    tol = ACC * (2 * uw + np.abs(W)) + 2.0 ** -22 * (uw + (0 if b is None else np.abs(B)))
    within(y, ref, U[dt] * np.abs(ref) + tol + TINY[dt], "y")
    # gradients, at the stored h with the forward's mean and rstd
    dy, dh = strided(randn(5, (rows, cols), dt), pad, 1 if pad else 0), randn(6, (rows, cols), dt)
    dx, dw, db = dion.layernorm_backward(dy, h, w, mean, rstd, dh=dh if residual else None, bias=bias)
    DY, H, M, R = n64(dy), n64(h), n64(mean), n64(rstd)
    dxr, dwr, dbr = O.layernorm_backward(DY, H, W, M, R, n64(dh) if residual else None)
    v, g = (H - M[:, None]) * R[:, None], DY * W
    t = ACC * R[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True) +
                            np.abs(v) * np.abs(g * v).mean(1, keepdims=True))
    within(dx, dxr, U[dt] * np.abs(dxr) + t + TINY[dt], "dx")
    within(dw, dwr, U[wd] * np.abs(dwr) + ACC * np.abs(DY * v).sum(0) + TINY[wd], "dw")
    if bias:
        within(db, dbr, U[wd] * np.abs(dbr) + ACC * np.abs(DY).sum(0) + TINY[wd], "db")
    else:
        assert db is None


def test_layernorm_gradient_against_differences(dion):
    """Directional central differences of the fp32 forward.  With unit-sized x, weights and directions of norm 1 and step
    e = 2^-4 the truncation is below e^2 |direction|^3 / 6 times third derivatives of order one, under 1e-3, and the
    rounding of y (2^-24 relative, 200 terms of order one) over 2e below 200 * 2^-24 * 8 = 1e-4: 2e-3 in all."""
    rows, cols, e = 2, 100, 2.0 ** -4
    x, dy, v = (randn(i, (rows, cols), torch.float32) for i in (11, 12, 13))
    v = v / v.norm()
    w, b = 1 + 0.3 * randn(14, (cols,), torch.float32), randn(16, (cols,), torch.float32)
    y, h, mean, rstd = dion.layernorm(x, w, b)
    dx, dw, db = dion.layernorm_backward(dy, h, w, mean, rstd)
    f = lambda *t: float((dion.layernorm(*t)[0].double() * dy.double()).sum())
    assert abs((f(x + e * v, w, b) - f(x - e * v, w, b)) / (2 * e) - float((dx * v).double().sum())) <= 2e-3
    u = randn(15, (cols,), torch.float32)
    u = u / u.norm()
    assert abs((f(x, w + e * u, b) - f(x, w - e * u, b)) / (2 * e) - float((dw * u).double().sum())) <= 2e-3
    assert abs((f(x, w, b + e * u) - f(x, w, b - e * u)) / (2 * e) - float((db * u).double().sum())) <= 2e-3


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 1000, 5003])
@pytest.mark.parametrize("cols", [3, 96, 520, 9000])
def test_layernorm_weight_gradients_over_many_rows(dion, rows, cols):
    x, dy = randn(6, (rows, cols), torch.bfloat16), randn(7, (rows, cols), torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    _, h, mean, rstd = dion.layernorm(x, w)
    dx, dw, db = dion.layernorm_backward(dy, h, w, mean, rstd)
    terms = n64(dy) * (n64(h) - n64(mean)[:, None]) * n64(rstd)[:, None]
    within(dw, terms.sum(0), ACC * np.abs(terms).sum(0) + 1e-30, "dw")
    within(db, n64(dy).sum(0), ACC * np.abs(n64(dy)).sum(0) + 1e-30, "db")
    for a, b in zip(dion.layernorm_backward(dy, h, w, mean, rstd), (dx, dw, db)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [40, 1000, 30000])
def test_layernorm_rows_far_from_zero(dion, cols):
    """A mean of 2^14 with a spread of 1: the differences are exact (both are multiples of 2^-9), so that nothing but
    the usual tolerance is lost; integers and halves around it are exact in fp32."""
    x = (randn(21, (6, cols), torch.float32) * 64).round() / 64 + 16384
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    y, _, mean, rstd = dion.layernorm(x, w, b, eps=1e-5)
    ref, mref, rref = O.layernorm(n64(x), n64(w), n64(b), 1e-5)
    within(rstd, rref, 2 * ACC * rref, "rstd")
    within(y, ref, ACC * (2 * np.abs(ref) + 1) + 2.0 ** -22 * np.abs(ref), "y")


def test_layernorm_special_rows(dion):
    """Rows of equal elements, and rows with an infinity or a NaN: the others do not see them."""
    for dtype in (torch.bfloat16, torch.float32):
        for cols in (200, 40000):
            x = randn(8, (6, cols), dtype)
            x[1] = 3
            x[3, 7] = float("inf")
            x[4, cols - 1] = float("nan")
            w, b = randn(9, (cols,), dtype), randn(10, (cols,), dtype)
            y, _, mean, rstd = dion.layernorm(x, w, b, eps=0.01)
            assert torch.equal(y[1], b) and mean[1] == 3 and torch.isnan(y[3:5]).all()
            clean = dion.layernorm(x[[0, 2, 5]], w, b, eps=0.01)
            assert torch.equal(y[[0, 2, 5]], clean[0]) and torch.equal(mean[[0, 2, 5]], clean[2])


# --------------------------------------------------- microscaled 4-bit codes
@pytest.mark.parametrize("rows,cols", [(0, 8), (1, 1), (1, 2), (3, 5), (2, 31), (2, 32), (7, 33), (40, 129), (7, 4096),
                                       (2, 30001), (300, 64), (1, 70000), (513, 777)])
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("fp16", 3), ("fp32", 4)])
def test_mxfp4_codes_are_the_definition(dion, rows, cols, dtype, pad):
    x = randn(21, (rows, cols), DT[dtype]) * (10.0 ** torch.randint(-4, 5, (rows, 1), generator=gen(3), device="cuda"))
    x = strided(x.to(DT[dtype]), pad if rows else 0, 1)
    q, scale = dion.mxfp4_quantize(x)
    assert q.dtype == scale.dtype == torch.uint8
    code, sref = O.mx_codes(n64(x))
    assert np.array_equal(scale.cpu().numpy(), sref)
    assert np.array_equal(q.cpu().numpy(), O.mx_pack(code))
    for out in (torch.bfloat16, torch.float16, torch.float32):
        y = dion.mxfp4_dequantize(q, scale, out, cols=cols)
        want = torch.from_numpy(O.mx_values(q.cpu().numpy(), sref, cols))
        assert torch.equal(y.cpu(), want.float().to(out))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_mxfp4_codes_at_the_borders(dion, dtype):
    """Every border between two codes and its neighbours in the type, at scales over the type's range, each as the
    largest of its block and below it; zeros of both signs; the largest and smallest values."""
    dt = DT[dtype]
    info = torch.finfo(dt)
    borders = torch.tensor([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 8], dtype=torch.float64)
    lo, hi = (-149 if dtype == "fp32" else -133 if dtype == "bf16" else -24), (125 if dtype != "fp16" else 12)
    values = torch.cat([borders * 2.0 ** e for e in range(lo, hi)])
    values = values[values <= info.max].to(dt)
    nudge = torch.nextafter if dtype == "fp32" else None
    if nudge:
        values = torch.cat([values, nudge(values, torch.zeros(())), nudge(values, torch.full((), info.max))])
    else:   # neighbours by their bit patterns
        bits = values.view(torch.int16)
        values = torch.cat([values, (bits - 1).clamp_min(0).view(dt), (bits + 1).view(dt)])
        values = values[torch.isfinite(values)]
    rows = []
    for top in (0.0, 4.0, 6.0):   # alone, or below a block's largest of 4 or 6 times its power of two
        x = torch.zeros(len(values), 32, dtype=dt)
        x[:, 3] = values
        x[:, 4] = -values
        if top:
            e = torch.floor(torch.log2(values.double().clamp_min(2.0 ** -149)))
            x[:, 9] = (top * 2.0 ** e.clamp_max(hi - 2)).to(dt)
        x[:, 31] = -0.0
        rows.append(x)
    x = torch.cat(rows).cuda()
    q, scale = dion.mxfp4_quantize(x)
    code, sref = O.mx_codes(n64(x))
    assert np.array_equal(scale.cpu().numpy(), sref)
    assert np.array_equal(q.cpu().numpy(), O.mx_pack(code))


def test_mxfp4_special_blocks(dion):
    """A block with an infinity or a NaN reads back as NaN; its neighbours do not see it."""
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x = randn(5, (4, 100), dtype)
        clean = dion.mxfp4_dequantize(*dion.mxfp4_quantize(x), dtype)
        x[1, 40] = float("inf")
        x[2, 99] = float("nan")
        q, scale = dion.mxfp4_quantize(x)
        y = dion.mxfp4_dequantize(q, scale, dtype)
        assert scale[1, 1] == 255 and scale[2, 3] == 255 and not q[1, 16:32].any() and not q[2, 48:].any()
        assert torch.isnan(y[1, 32:64]).all() and torch.isnan(y[2, 96:]).all()
        y[1, 32:64], y[2, 96:] = clean[1, 32:64], clean[2, 96:]
        assert torch.equal(y, clean)


# ------------------------------------------------------------- 4-bit product
def mx_matrix(seed, rows, k, pad=0):
    """Any codes with scales around one, their values in float64, and both in rows further apart."""
    g = gen(seed)
    q = torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda").to(torch.uint8)
    s = torch.randint(120, 131, (rows, (k + 31) // 32), generator=g, device="cuda").to(torch.uint8)
    v = O.mx_values(q.cpu().numpy(), s.cpu().numpy(), k)
    return strided(q, pad, pad // 2), strided(s, pad, pad // 3), v


def mx_tolerance(A, B, prod, bias, k, dt):
    mag = np.abs(A) @ np.abs(B).T
    total = prod + bias
    return U[dt] * np.abs(total) + (k / 64 + 80) * 2.0 ** -23 * mag + 2.0 ** -23 * (np.abs(prod) + np.abs(bias)) + TINY[dt]


LINEAR = [(1, 1, 2), (1, 5, 0), (2, 3, 18), (1, 64, 64), (1, 1000, 334), (3, 257, 128), (5, 31, 4096), (16, 96, 640),
          (17, 100, 300), (24, 520, 1024), (33, 129, 66), (64, 256, 2048), (65, 300, 510), (100, 64, 14336),
          (128, 128, 256), (129, 257, 200), (200, 1000, 778), (256, 512, 1024), (300, 270, 130), (515, 777, 640),
          (1030, 260, 384), (70, 90, 48), (300, 140, 208), (1500, 1300, 1040), (4100, 4200, 400), (1, 14000, 512),
          (7, 14001, 1000), (3000, 3001, 1536), (2, 100, 14336), (40, 40, 32), (2049, 1793, 2560), (130, 130, 512), (40, 70, 0), (9, 14336, 768)]


@pytest.mark.parametrize("m,n,k", LINEAR)
@pytest.mark.parametrize("out,bias,pad", [("bf16", None, 0), ("fp32", "fp32", 5), ("fp16", "bf16", 16)])
def test_mxfp4_linear(dion, m, n, k, out, bias, pad):
    a, sa, A = mx_matrix(m * 7 + k, m, k, pad if k else 0)
    b, sb, B = mx_matrix(n * 3 + k + 1, n, k, pad if k else 0)
    bv = None if bias is None else randn(5, (n,), DT[bias])
    y = dion.mxfp4_linear(a, sa, b, sb, bias=bv, out_dtype=DT[out])
    assert y.shape == (m, n) and y.dtype == DT[out]
    prod, bb = A @ B.T, 0 if bias is None else n64(bv)
    tol = mx_tolerance(A, B, prod, bb, k, DT[out])
    if out == "fp16":   # beyond its range it is infinite
        prod = np.where(np.abs(prod + bb) < 65520, prod, np.copysign(np.inf, prod))
    within(y, prod + bb, tol, "out")
    again = dion.mxfp4_linear(a, sa, b, sb, bias=bv, out_dtype=DT[out])
    assert torch.equal(again, y)


@pytest.mark.parametrize("m,n,k", [(1, 48, 512), (9, 70, 2048), (40, 64, 512), (130, 200, 1024), (600, 700, 512),
                                   (1300, 1100, 544)])
def test_mxfp4_linear_places_every_element(dion, m, n, k):
    """One element of a and one of b at a time in each pair of rows: the product says where they met.  All sums are
    exact, so the outputs are too."""
    rng = np.random.default_rng(m + n + k)
    ca, cb = np.zeros((m, k), np.uint8), np.zeros((n, k), np.uint8)
    at_a, at_b = rng.integers(0, k, m), rng.integers(0, k, n)
    at_b[::3] = at_a[rng.integers(0, m, len(at_b[::3]))]
    ca[np.arange(m), at_a] = rng.integers(1, 16, m)
    cb[np.arange(n), at_b] = rng.integers(1, 16, n)
    sa, sb = (rng.integers(110, 140, (r, (k + 31) // 32)).astype(np.uint8) for r in (m, n))
    qa, qb = O.mx_pack(ca), O.mx_pack(cb)
    want = O.mx_values(qa, sa, k) @ O.mx_values(qb, sb, k).T
    put = lambda v: torch.from_numpy(v).cuda()
    y = dion.mxfp4_linear(put(qa), put(sa), put(qb), put(sb), out_dtype=torch.float32)
    assert np.array_equal(n64(y), want) and np.count_nonzero(want) >= n // 4


@pytest.mark.parametrize("m", [1, 16, 17, 200, 1030])
def test_mxfp4_linear_nan_scales_stay_in_their_rows(dion, m):
    k, n = 640, 300
    a, sa, A = mx_matrix(1, m, k)
    b, sb, B = mx_matrix(2, n, k)
    clean = dion.mxfp4_linear(a, sa, b, sb, out_dtype=torch.float32)
    sb[37, 11] = 255
    sa[m - 1, 19] = 255
    y = dion.mxfp4_linear(a, sa, b, sb, out_dtype=torch.float32)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[:, 37] = True
    bad[m - 1] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("m,n", [(1, 37), (16, 21), (40, 70), (300, 333)])
@pytest.mark.parametrize("k,gap", [(10, 2), (254, 0), (256, 1), (258, 3), (1024, 5), (4098, 0)])
@pytest.mark.parametrize("start", [0, 1, 4])
def test_mxfp4_linear_rows_at_any_byte(dion, m, n, k, gap, start):
    """Codes and scales at any byte, between other bytes (NaN scales among them) that must not count."""
    def put(v):
        rows, cols = v.shape
        whole = torch.full((start + rows * (cols + gap),), 255, dtype=torch.uint8, device="cuda")
        t = whole[start:].view(rows, cols + gap)[:, :cols]
        t.copy_(v)
        return t
    a, sa, A = mx_matrix(3, m, k)
    b, sb, B = mx_matrix(4, n, k)
    y = dion.mxfp4_linear(put(a), put(sa), put(b), put(sb), out_dtype=torch.float32)
    prod = A @ B.T
    within(y, prod, mx_tolerance(A, B, prod, 0, k, torch.float32), "out")


def test_mxfp4_linear_leading_dimensions_and_odd_columns(dion):
    x, w = randn(1, (4, 10, 101), torch.bfloat16), randn(2, (70, 101), torch.bfloat16)
    (a, sa), (b, sb) = dion.mxfp4_quantize(x), dion.mxfp4_quantize(w)
    assert a.shape == (4, 10, 51) and sa.shape == (4, 10, 4)
    y = dion.mxfp4_linear(a, sa, b, sb, out_dtype=torch.float32)
    A = n64(dion.mxfp4_dequantize(a, sa, torch.float32, cols=101)).reshape(40, 101)
    B = n64(dion.mxfp4_dequantize(b, sb, torch.float32, cols=101))
    within(y.view(40, 70), A @ B.T, mx_tolerance(A, B, A @ B.T, 0, 102, torch.float32), "out")


# ----------------------------------------------------------- log probabilities
def logits_case(rows, vocab, dt, seed=0, spread=2.0):
    g = gen(seed + rows * 31 + vocab)
    z = (torch.randn((rows, vocab), generator=g, device="cuda") * spread).to(dt)
    tokens = torch.randint(vocab, (rows,), generator=g, device="cuda")
    if rows > 2:
        tokens[1], tokens[2] = -100, vocab
    return z, tokens


def logprob_check(dion, z, tokens, temp, k, gl, ge):
    dt = z.dtype
    rows, vocab = z.shape
    Z, T = n64(z), tokens.cpu().numpy()
    lp, ent, logq, q = O.logprobs(Z, T, temp)
    with np.errstate(all="ignore"):
        u = np.where(np.isfinite(Z), (Z - Z.max(1, keepdims=True)) / temp, 0)
        ls = np.log(np.exp(np.where(np.isfinite(Z), u, -np.inf)).sum(1, keepdims=True))
    ls = np.where(np.isfinite(ls), np.abs(ls), 0)
    D = np.abs(u) + ls + ent[:, None] + 4
    inside = (T >= 0) & (T < vocab)
    Dt = D[np.arange(rows), np.where(inside, T, 0)]
    got, gent, stats = dion.token_logprobs(z, tokens, temperature=temp)
    within(got, lp, ACC + 2.0 ** -21 * Dt, "logprob")
    near = ls[:, 0] + ent + 4   # what reaches the entropy: terms with a weight
    etol = (ACC + 2.0 ** -20 * near) * (1 + ent)
    within(gent, ent, etol, "entropy")
    if k:
        top, index, lp2, ent2 = dion.top_logprobs(z, k, tokens, temperature=temp)
        ref = O.top(Z, k)
        assert np.array_equal(index.cpu().numpy(), ref), "index"
        at = np.where(ref >= 0, ref, 0)
        want = np.where(ref >= 0, np.take_along_axis(logq, at, 1), -np.inf)
        within(top, want, ACC + 2.0 ** -21 * np.take_along_axis(D, at, 1), "top")
        within(lp2, lp, ACC + 2.0 ** -21 * Dt, "logprob beside the top")
        within(ent2, ent, etol, "entropy beside the top")
        more = dion.top_logprobs(z, k, temperature=temp)
        assert torch.equal(more[1], index) and torch.equal(more[0], top) and more[2] is None
    GL = np.zeros(rows) if gl is None else n64(gl)
    GE = np.zeros(rows) if ge is None else n64(ge)
    ref = O.logprobs_backward(GL, GE, Z, T, temp)
    hit = (np.arange(vocab) == T[:, None])
    tol = q * (ACC + 2.0 ** -20 * D) * (np.abs(GL)[:, None] + np.abs(GE)[:, None] * (1 + D))
    tol = (tol + 2.0 ** -22 * hit * np.abs(GL)[:, None]) / temp
    d = dion.token_logprobs_backward(gl, ge, z, stats, tokens, temperature=temp)
    assert d.shape == z.shape and d.dtype == dt
    within(d, ref, U[dt] * np.abs(ref) + tol + TINY[dt], "dlogits")
    zero = ((GL == 0) | ~inside) & (GE == 0)
    assert not n64(d)[zero].any()
    copy = z.clone()
    assert dion.token_logprobs_backward(gl, ge, copy, stats, tokens, temperature=temp, out=copy) is copy
    assert torch.equal(copy, d)


LOGPROB = [(1, 1, 1), (3, 2, 2), (1, 17, 5), (5, 1000, 1), (3, 1023, 64), (16, 4096, 100), (2, 50257, 20),
           (1, 131072, 128), (7, 32001, 17), (300, 257, 8), (20, 8192, 1024), (33, 40000, 3), (4, 32768, 256),
           (3, 32769, 257), (600, 2000, 40), (5, 131073, 1000), (3, 100, 1024), (2, 300000, 64), (260, 5000, 12),
           (1, 49152, 32), (32, 50000, 5), (33, 50000, 5), (3, 400001, 32), (17, 65537, 1), (1, 128256, 20)]


@pytest.mark.parametrize("rows,vocab,k", LOGPROB)
@pytest.mark.parametrize("dtype,temp,pad,ttype", [("bf16", 1.0, 0, torch.int64), ("fp32", 2.0, 7, torch.int32),
                                                  ("fp16", 0.5, 16, torch.int64)])
def test_logprobs(dion, rows, vocab, k, dtype, temp, pad, ttype):
    z, tokens = logits_case(rows, vocab, DT[dtype])
    gl, ge = randn(1, (rows,), torch.float32), randn(2, (rows,), torch.float32)
    gl[rows // 2] = 0
    ge[rows // 2:] = 0
    logprob_check(dion, strided(z, pad, pad // 2), tokens.to(ttype), temp, k, gl, ge)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_with_either_gradient_alone(dion, dtype):
    z, tokens = logits_case(9, 777, DT[dtype])
    one = torch.ones(9, device="cuda")
    for gl, ge in ((one, None), (None, one), (None, None)):
        logprob_check(dion, z, tokens, 1.0, 0, gl, ge)


@pytest.mark.parametrize("vocab", [500, 40001, 131072, 262145, 524288])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_top_of_equal_ascending_and_masked_rows(dion, vocab, dtype):
    """Rows of equal logits, few values, ascending and descending ones, with the largest side by side, at the ends, and
    with masks of -inf or the type's lowest value that leave little or nothing."""
    dt = DT[dtype]
    low = torch.finfo(dt).min
    g = gen(4)
    z = torch.zeros((14, vocab), device="cuda", dtype=dt)
    z[1] = torch.randint(0, 3, (vocab,), generator=g, device="cuda").to(dt)
    z[2] = torch.linspace(-8, 8, vocab, device="cuda").to(dt)
    z[3] = torch.linspace(8, -8, vocab, device="cuda").to(dt)
    z[4:8] = torch.randn((4, vocab), generator=g, device="cuda").to(dt)
    z[5, 100:180] += 9
    z[6, -40:] = 11
    z[7, :3] = 12
    z[8] = -float("inf")
    z[9] = -float("inf")
    z[9, [7, 8, vocab - 1]] = torch.tensor([1.0, 2.0, 1.0], device="cuda").to(dt)
    z[10] = low
    z[11] = low
    z[11, 11:400:7] = randn(6, (56,), dt)
    z[12] = -0.0
    z[12, ::2] = 0.0
    z[13] = torch.randint(-2, 1, (vocab,), generator=g, device="cuda").to(dt) * 1000
    tokens = torch.full((14,), 7, device="cuda")
    gl = torch.ones(14, device="cuda")
    for k in (1, 20, 64, 130):
        logprob_check(dion, z, tokens, 1.0, k, gl, -0.5 * gl)


@pytest.mark.parametrize("vocab", [300, 40000, 70000])
def test_logprobs_nan_and_infinite_rows(dion, vocab):
    """A NaN or +inf makes its row's statistics NaN, and no other's; a left-out row has gradient 0 whatever it holds."""
    z, _ = logits_case(5, vocab, torch.float32)
    z[1, 5] = float("nan")
    z[3, vocab - 1] = float("inf")
    tokens = torch.tensor([1, 2, 3, 4, -1], device="cuda")
    top, index, lp, ent = dion.top_logprobs(z, 9, tokens)
    assert torch.isnan(lp[[1, 3]]).all() and torch.isnan(ent[[1, 3]]).all() and torch.isnan(top[[1, 3]]).all()
    ref = O.top(np.nan_to_num(n64(z), nan=-np.inf, posinf=1e300), 9)
    assert np.array_equal(index.cpu().numpy(), ref)
    clean = dion.top_logprobs(z[[0, 2, 4]], 9, tokens[[0, 2, 4]])
    for a, b in zip((top, index, lp, ent), clean):
        assert torch.equal(a[[0, 2, 4]], b)
    stats = dion.token_logprobs(z, tokens)[2]
    gl = torch.tensor([1.0, 0, 1, 1, 1], device="cuda")
    d = dion.token_logprobs_backward(gl, None, z, stats, tokens)
    assert torch.isnan(d[3]).all() and not d[1].any() and not d[4].any() and torch.isfinite(d[[0, 2]]).all()


@pytest.mark.parametrize("shift", [0.0, 30000.0, -60000.0])
@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_logprobs_far_from_zero(dion, shift, dtype):
    z, tokens = logits_case(6, 3001, torch.float32)
    z = ((z * 16).round() / 16 + shift).to(DT[dtype])
    one = torch.ones(6, device="cuda")
    logprob_check(dion, z, tokens, 1.0, 11, one, one)


def test_logprobs_of_nearly_certain_rows_keep_a_small_entropy(dion):
    """One logit 20 above 1000 others: a mass of 2e-6 and an entropy of 4.3e-5, of which 2e-6 is log s and the rest the
    others' share.  s = 1 + 2e-6 is off by 2^-24 for each of the at most 12 additions that its 1 goes through."""
    z = torch.zeros((3, 1001), device="cuda")
    z[:, 500] = 20.0
    _, ent, _ = dion.token_logprobs(z, torch.zeros(3, dtype=torch.int64, device="cuda"))
    _, ref, _, _ = O.logprobs(n64(z), np.zeros(3, np.int64), 1.0)
    within(ent, ref, 12 * 2.0 ** -24 + ref * 2.0 ** -14, "entropy")


# ------------------------------------------------------ beyond 2^31 elements
def test_offsets_beyond_32_bits(dion):
    """Rows behind 2^31 elements (and 2^32 bytes) come out as they do alone."""
    rows, cols = 300000, 8192
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    x[-3:] = randn(1, (3, cols), torch.bfloat16)
    tail = x[-3:].clone()
    w, b = randn(2, (cols,), torch.bfloat16), randn(3, (cols,), torch.bfloat16)
    y, _, mean, rstd = dion.layernorm(x, w, b)
    ty, _, tmean, trstd = dion.layernorm(tail, w, b)
    assert torch.equal(y[-3:], ty) and torch.equal(mean[-3:], tmean) and torch.equal(rstd[-3:], trstd)
    dx, _, _ = dion.layernorm_backward(y, x, w, mean, rstd)
    assert torch.equal(dx[-3:], dion.layernorm_backward(ty, tail, w, tmean, trstd)[0])
    del y, dx
    q, s = dion.mxfp4_quantize(x)
    tq, ts = dion.mxfp4_quantize(tail)
    assert torch.equal(q[-3:], tq) and torch.equal(s[-3:], ts)
    back = dion.mxfp4_dequantize(q, s)
    assert torch.equal(back[-3:], dion.mxfp4_dequantize(tq, ts))
    del back
    # a product whose output and first operand are as large
    head, hs = dion.mxfp4_quantize(randn(4, (8000, cols), torch.bfloat16))
    out = dion.mxfp4_linear(q, s, head, hs)
    want = dion.mxfp4_linear(q[-256:].contiguous(), s[-256:].contiguous(), head, hs, out_dtype=torch.float32)
    assert not out[:5].any()
    ref = n64(want[-3:])
    within(out[-3:], ref, 2.0 ** -8 * np.abs(ref) + (cols / 64 + 80) * 2.0 ** -22 * np.abs(ref).max(), "out")
    del out, q, s, want
    t = torch.arange(rows, device="cuda") % cols
    lp, ent, stats = dion.token_logprobs(x, t)
    top, index, lp2, _ = dion.top_logprobs(x, 4, t)
    a = dion.token_logprobs(tail, t[-3:])
    c = dion.top_logprobs(tail, 4, t[-3:])
    assert torch.equal(lp, lp2) and torch.equal(index[-3:], c[1])
    within(lp[-3:], n64(a[0]), 2.0 ** -18, "logprob")   # 256 threads against 1024: the same to a few roundings of 10
    one = torch.ones(rows, device="cuda")
    d = dion.token_logprobs_backward(one, None, x, stats, t)
    e = dion.token_logprobs_backward(one[-3:], None, tail, stats[-3:].contiguous(), t[-3:])
    assert torch.equal(d[-3:], e)


# ------------------------------------------------- streams, graphs, autograd
def run_of_them(dion, x, res, w, b, head, head_s, z, index_k=16):
    """The operators as a distillation step uses them: norm, codes, product with the teacher's head, its top entries,
    the student's loss on them, log probabilities and gradients."""
    y, h, mean, rstd = dion.layernorm(x, w, b, residual=res)
    q, s = dion.mxfp4_quantize(y)
    logits = dion.mxfp4_linear(q, s, head, head_s, out_dtype=torch.float32)
    top, index, _, ent = dion.top_logprobs(logits, index_k)
    loss, dz = dion.distill_topk_step(z, top, index)
    lp, e2, stats = dion.token_logprobs(z, index[:, 0])
    dlp = dion.token_logprobs_backward(torch.ones_like(lp), None, z, stats, index[:, 0])
    dx, dw, db = dion.layernorm_backward(y, h, w, mean, rstd)
    return y, h, q, s, logits, top, index, ent, loss, dz, lp, e2, dlp, dx, dw, db


def step_inputs(dion, tokens=200, dim=160, vocab=1500):
    x, res = randn(1, (tokens, dim), torch.bfloat16), randn(2, (tokens, dim), torch.bfloat16)
    w, b = randn(3, (dim,), torch.bfloat16), randn(4, (dim,), torch.bfloat16)
    head, head_s = dion.mxfp4_quantize(randn(5, (vocab, dim), torch.bfloat16))
    return x, res, w, b, head, head_s, randn(6, (tokens, vocab), torch.bfloat16)


def test_a_run_of_them_agrees_with_the_oracle(dion):
    x, res, w, b, head, head_s, z = step_inputs(dion)
    y, h, q, s, logits, top, index, ent, loss, dz, lp, e2, dlp, dx, dw, db = run_of_them(
        dion, x, res, w, b, head, head_s, z)
    code, scale = O.mx_codes(n64(y))   # from the norm's output on, each from what it was given
    assert np.array_equal(q.cpu().numpy(), O.mx_pack(code)) and np.array_equal(s.cpu().numpy(), scale)
    A, B = O.mx_values(O.mx_pack(code), scale, 160), O.mx_values(head.cpu().numpy(), head_s.cpu().numpy(), 160)
    within(logits, A @ B.T, mx_tolerance(A, B, A @ B.T, 0, 160, torch.float32), "logits")
    assert np.array_equal(index.cpu().numpy(), O.top(n64(logits), 16))
    ref, refent, _, _ = O.logprobs(n64(logits), index[:, 3].cpu().numpy(), 1.0)
    within(top[:, 3], ref, ACC + 2.0 ** -19 * (np.abs(ref) + 12), "top")
    ref, _, _, _ = O.logprobs(n64(z), index[:, 0].cpu().numpy(), 1.0)
    within(lp, ref, ACC + 2.0 ** -20 * (np.abs(ref) + 12), "logprob")
    # the loss on entries given as log probabilities is the loss on the logits themselves: the difference is a constant
    loss2, _ = dion.distill_topk_step(z, logits.gather(1, index), index)
    within(loss, n64(loss2), 2 * (ACC + 2.0 ** -21 * 60), "loss")


def test_a_run_of_them_on_another_stream_and_in_a_graph(dion):
    args = step_inputs(dion)
    want = [t.clone() for t in run_of_them(dion, *args)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_of_them(dion, *args)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_of_them(dion, *args)
    for i in range(3):
        for t in out:
            t.zero_()
        eager = run_of_them(dion, *args)   # the program's own work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(out, want, eager):
            assert torch.equal(a, b) and torch.equal(c, b), i


def test_the_stream_argument(dion):
    x, res, w, b, head, head_s, z = step_inputs(dion, 64, 96, 700)
    want = run_of_them(dion, x, res, w, b, head, head_s, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, mean, rstd = dion.layernorm(x, w, b, residual=res, stream=side)
    q, s = dion.mxfp4_quantize(y, stream=side)
    logits = dion.mxfp4_linear(q, s, head, head_s, out_dtype=torch.float32, stream=side)
    top, index, _, ent = dion.top_logprobs(logits, 16, stream=side)
    back = dion.mxfp4_dequantize(q, s, stream=side)
    side.synchronize()
    first = index[:, 0]   # not contiguous: copied on the stream
    lp, e2, stats = dion.token_logprobs(z, first, stream=side)
    dlp = dion.token_logprobs_backward(torch.ones(64, device="cuda"), None, z, stats, first, stream=side)
    dx, dw, db = dion.layernorm_backward(y, h, w, mean, rstd, stream=side)
    side.synchronize()
    got = (y, h, q, s, logits, top, index, ent, want[8], want[9], lp, e2, dlp, dx, dw, db)
    for i, (a, c) in enumerate(zip(got, want)):
        assert torch.equal(a, c), i
    assert torch.equal(back, dion.mxfp4_dequantize(q, s))


def test_autograd(dion):
    x, res, w, b, _, _, _ = step_inputs(dion, 40, 64, 300)
    for dtype in (torch.float32, torch.bfloat16):
        leaf = lambda t: t.to(dtype).clone().requires_grad_()
        X, R, Wt, Bt = leaf(x), leaf(res), leaf(w), leaf(b)
        y, h = dion.layer_norm(X, Wt, Bt, R)
        gy, gh = randn(1, y.shape, dtype), randn(2, y.shape, dtype)
        torch.autograd.backward((y, h), (gy, gh))
        want = dion.layernorm_backward(gy, *[dion.layernorm(X.detach(), Wt.detach(), Bt.detach(), R.detach())[i]
                                             for i in (1,)], Wt.detach(),
                                       *dion.layernorm(X.detach(), Wt.detach(), Bt.detach(), R.detach())[2:], dh=gh)
        assert torch.equal(X.grad, want[0]) and torch.equal(R.grad, want[0])
        assert torch.equal(Wt.grad, want[1]) and torch.equal(Bt.grad, want[2])
        # without a bias or a residual, from a transposed input; only the residual stream used
        X2 = leaf(x)
        dion.layer_norm(X2.t().contiguous().t(), Wt.detach().requires_grad_()).sum().backward()
        assert torch.isfinite(X2.grad).all()
        X3, R3 = leaf(x), leaf(res)
        dion.layer_norm(X3, Wt.detach(), Bt.detach(), R3)[1].sum().backward()
        assert torch.equal(X3.grad, torch.ones_like(X3)) and torch.equal(R3.grad, torch.ones_like(R3))
        # log probabilities: both outputs, one of them, and a broadcast gradient
        Z = leaf(randn(3, (40, 300), torch.float32))
        t = torch.arange(40, device="cuda")
        lp, ent = dion.log_probs(Z, t, 0.5)
        (lp.sum() + 0.25 * ent.sum()).backward()
        one = torch.ones(40, device="cuda")
        stats = dion.token_logprobs(Z.detach(), t, 0.5)[2]
        assert torch.equal(Z.grad, dion.token_logprobs_backward(one, 0.25 * one, Z.detach(), stats, t, 0.5))
        Z2 = leaf(randn(3, (40, 300), torch.float32))
        dion.log_probs(Z2.t().contiguous().t(), t, 0.5)[0].sum().backward()
        assert torch.equal(Z2.grad, dion.token_logprobs_backward(one, None, Z.detach(), stats, t, 0.5))


def test_a_second_differentiation_raises(dion):
    x = randn(1, (4, 32), torch.float32).requires_grad_()
    w = torch.ones(32, device="cuda", requires_grad=True)
    b = torch.zeros(32, device="cuda", requires_grad=True)
    t = torch.arange(4, device="cuda")
    for out in (dion.layer_norm(x, w, b), dion.log_probs(x, t)[0], dion.log_probs(x, t)[1]):
        (g,) = torch.autograd.grad(out.sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiate twice"):
            g.sum().backward()


def test_refusals(dion):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    q, s = dion.mxfp4_quantize(x)
    z, t = torch.zeros(4, 50, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    stats = dion.token_logprobs(z, t)[2]
    one = torch.ones(4, device="cuda")
    calls = [
        lambda: dion.layernorm(x.cpu(), w), lambda: dion.layernorm(x, w.half()), lambda: dion.layernorm(x, w, w.float()),
        lambda: dion.layernorm(x, w[:32]), lambda: dion.layernorm(x, w, residual=x[:2]),
        lambda: dion.layernorm(x, w, residual=x.float()), lambda: dion.layernorm(x.t(), w),
        lambda: dion.layernorm(x, w, eps=-1.0), lambda: dion.layernorm(x.to(torch.float64), w),
        lambda: dion.layernorm(torch.zeros(1, 70000, device="cuda"), torch.ones(70000, device="cuda")),
        lambda: dion.layernorm_backward(x, x, w, one[:2], one), lambda: dion.layernorm_backward(x[:2], x, w, one, one),
        lambda: dion.layernorm_backward(x, x, w, one, one, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")),
        lambda: dion.mxfp4_quantize(x.long()), lambda: dion.mxfp4_quantize(x[:, :0]),
        lambda: dion.mxfp4_dequantize(q.to(torch.int8), s), lambda: dion.mxfp4_dequantize(q, s[:, :1]),
        lambda: dion.mxfp4_dequantize(q, s, cols=62), lambda: dion.mxfp4_dequantize(q, s, torch.int8),
        lambda: dion.mxfp4_linear(q, s, q[:, :16], s[:, :1]), lambda: dion.mxfp4_linear(q, s, q, s[:2]),
        lambda: dion.mxfp4_linear(q, s, q, s.cpu()), lambda: dion.mxfp4_linear(q, s, q, s, bias=w),
        lambda: dion.mxfp4_linear(q, s, q, s, out_dtype=torch.int8), lambda: dion.mxfp4_linear(q, s, q[None], s[None]),
        lambda: dion.token_logprobs(z, t[:3]), lambda: dion.token_logprobs(z, t.float()),
        lambda: dion.token_logprobs(z, None), lambda: dion.token_logprobs(z, t, temperature=0.0),
        lambda: dion.token_logprobs(z.t(), torch.zeros(50, dtype=torch.int64, device="cuda")),
        lambda: dion.top_logprobs(z, -1), lambda: dion.top_logprobs(z, 1025),
        lambda: dion.top_logprobs(torch.zeros(1, (1 << 19) + 1, device="cuda"), 1),
        lambda: dion.token_logprobs_backward(one[:2], None, z, stats, t),
        lambda: dion.token_logprobs_backward(one, None, z, stats[:2], t),
        lambda: dion.token_logprobs_backward(one, None, z, stats, t, out=z[:2]),
        lambda: dion.token_logprobs_backward(one, None, z, stats, t, out=z.half()),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(dion.DionError):
            call()
            print("not refused:", i)


def test_no_rows(dion):
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, h, mean, rstd = dion.layernorm(x, w, w)
    dx, dw, db = dion.layernorm_backward(y, x, w, mean, rstd)
    assert y.shape == dx.shape == (0, 64) and not dw.any() and not db.any()
    q, s = dion.mxfp4_quantize(x)
    b, sb = dion.mxfp4_quantize(torch.ones(5, 64, device="cuda"))
    assert q.shape == (0, 32) and dion.mxfp4_dequantize(q, s).shape == (0, 64)
    assert dion.mxfp4_linear(q, s, b, sb).shape == (0, 5) and dion.mxfp4_linear(b, sb, q, s).shape == (5, 0)
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    lp, ent, stats = dion.token_logprobs(x, t)
    assert lp.shape == (0,) and dion.top_logprobs(x, 3)[1].shape == (0, 3)
    assert dion.token_logprobs_backward(lp, ent, x, stats, t).shape == (0, 64)
