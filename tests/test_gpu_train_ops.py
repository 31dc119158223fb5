"""The training-step operators on the GPU against the float64 oracle.

Tolerances.  u is the largest relative rounding error of the output's type (bf16
2^-8, fp16 2^-11, fp32 2^-24).  An fp32 sum of n terms in which no partial sum runs over
more than 512 terms and a tree of 16 is off by at most 528 * 2^-24 < 2^-14 of
the sum of magnitudes; rounding errors are that large only if all of them
point one way.  ACC = 2^-15 allows half of it.
  norm       y, rstd        (u + ACC) |y|
  codes      |q scale - y|  <= (0.5 + 127 ACC) scale; scale itself ACC
  gradient   dx             u |dx| + ACC rstd (|g| + |h| rstd^2 mean|g h|)
             dw             u |dw| + ACC sum |dy h| rstd
  product    u |out| + 2^-22 (|product| + |bias|) (three fp32 roundings)
  loss       T^2 (ACC + 2^-21 D), D the largest magnitude of the exponents
             (z - max) / T and (t - max) / T and of the logarithm of the sum
             that enter it
  dlogits    u |dz| + |gl| T (q (ACC + 2^-21 D_j) + 2^-20 P_j), D_j = |z_j - max| / T + the logarithm
fp16 results below its normal range round to multiples of 2^-24: 2^-25 is added.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import train_oracle as O  # noqa: E402

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


def randn(seed, shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, ref, tol, what):
    got = n64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))))


# ------------------------------------------------------------------ RMS norm
NORM_SHAPES = [(1, 1), (3, 2), (2, 7), (5, 63), (4, 64), (17, 65), (130, 128), (9, 257), (65, 768), (33, 1001),
               (1, 4096), (3, 4097), (2, 8192), (2, 16384), (2, 20001), (1, 65536), (700, 100)]


def norm_case(rows, cols, dt, wdt, residual, pad):
    x = strided(randn(1, (rows, cols), dt), pad, pad // 2)
    r = strided(randn(2, (rows, cols), dt, 3.0), pad, pad // 3) if residual else None
    w = (1 + 0.3 * randn(3, (cols,), torch.float32)).to(wdt)
    return x, r, w


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype,wtype,residual,pad", [("bf16", "bf16", True, 0), ("fp16", "fp32", False, 3),
                                                      ("fp32", "fp32", True, 5), ("bf16", "fp32", True, 16),
                                                      ("fp16", "fp16", True, 0), ("fp32", "fp32", False, 0)])
def test_rmsnorm_forward_backward(dion, rows, cols, dtype, wtype, residual, pad):
    dt, eps = DT[dtype], 1e-5
    x, r, w = norm_case(rows, cols, dt, DT[wtype], residual, pad)
    s = x.float() + r.float() if residual else x.float()
    y, h, rstd = dion.rmsnorm(x, w, residual=r, eps=eps)
    assert torch.equal(h, s.to(dt))
    ref, rref = O.rmsnorm(n64(s), n64(w), eps)
    within(rstd, rref, ACC * rref, "rstd")
    within(y, ref, (U[dt] + ACC) * np.abs(ref) + TINY[dt], "y")
    # 8-bit codes of the same norm
    q, scale, h8 = dion.rmsnorm_int8(x, w, residual=r, eps=eps)
    assert torch.equal(h8, h) and q.dtype == torch.int8
    step = np.abs(ref).max(1) / 127
    within(scale, step, ACC * step, "scale")
    within(n64(q) * step[:, None], ref, (0.5 + 127 * ACC) * step[:, None], "codes")
    assert (n64(q).__abs__().max(1) == 127).all()
    # gradients
    dy, dh = strided(randn(4, (rows, cols), dt), pad, 1 if pad else 0), randn(5, (rows, cols), dt)
    dx, dw = dion.rmsnorm_backward(dy, h, w, rstd, dh=dh if residual else None)
    H, DY, W = n64(h), n64(dy), n64(w)
    # the gradient is taken at the stored h with the forward's rstd
    rs = n64(rstd)[:, None]
    g = DY * W
    dxr = rs * (g - H * (g * H).mean(1, keepdims=True) * rs ** 2) + (n64(dh) if residual else 0)
    tol = rs * (np.abs(g) + np.abs(H) * rs ** 2 * np.abs(g * H).mean(1, keepdims=True)) * ACC
    within(dx, dxr, U[dt] * np.abs(dxr) + tol + TINY[dt], "dx")
    dwr = (DY * H * rs).sum(0)
    wd = DT[wtype]
    within(dw, dwr, U[wd] * np.abs(dwr) + ACC * np.abs(DY * H * rs).sum(0) + TINY[wd], "dw")
    if dt == torch.float32:   # and is the definition's where h is not rounded
        dx64, dw64 = O.rmsnorm_backward(DY, H, W, eps, n64(dh) if residual else None)
        within(dx, dx64, 4 * tol + 1e-30 + ACC * np.abs(dx64), "dx by definition")
        within(dw, dw64, 4 * ACC * np.abs(DY * H * rs).sum(0), "dw by definition")


def test_rmsnorm_gradient_against_differences(dion):
    """Directional central differences of the fp32 forward.  With unit-sized x,
    weights and directions of norm 1 and step e = 2^-4 the truncation is below
    e^2 |direction|^3 / 6 times third derivatives of order one, under 1e-3, and
    the rounding of y (2^-24 relative, 200 terms of order one) over 2e below
    200 * 2^-24 * 8 = 1e-4: 2e-3 in all."""
    rows, cols, e = 2, 100, 2.0 ** -4
    x, dy, v = (randn(i, (rows, cols), torch.float32) for i in (11, 12, 13))
    v = v / v.norm()
    w = 1 + 0.3 * randn(14, (cols,), torch.float32)
    y, h, rstd = dion.rmsnorm(x, w)
    dx, dw = dion.rmsnorm_backward(dy, h, w, rstd)
    f = lambda t: float((dion.rmsnorm(t, w)[0].double() * dy.double()).sum())
    assert abs((f(x + e * v) - f(x - e * v)) / (2 * e) - float((dx * v).double().sum())) <= 2e-3
    u = randn(15, (cols,), torch.float32)
    u = u / u.norm()
    f = lambda t: float((dion.rmsnorm(x, t)[0].double() * dy.double()).sum())
    assert abs((f(w + e * u) - f(w - e * u)) / (2 * e) - float((dw * u).double().sum())) <= 2e-3


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 1000, 5003])
@pytest.mark.parametrize("cols", [3, 96, 520])
def test_rmsnorm_dweight_over_many_rows(dion, rows, cols):
    x, dy = randn(6, (rows, cols), torch.bfloat16), randn(7, (rows, cols), torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    _, h, rstd = dion.rmsnorm(x, w)
    dx, dw = dion.rmsnorm_backward(dy, h, w, rstd)
    terms = n64(dy) * n64(h) * n64(rstd)[:, None]
    within(dw, terms.sum(0), ACC * np.abs(terms).sum(0) + 1e-30, "dw")
    again = dion.rmsnorm_backward(dy, h, w, rstd)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_rmsnorm_special_rows(dion):
    """Zero rows, tiny rows, and rows with an infinity or a NaN: the others do not see them."""
    for dtype in (torch.bfloat16, torch.float32):
        x = randn(8, (6, 200), dtype)
        x[1] = 0
        x[2] *= 1e-20
        x[3, 7] = float("inf")
        x[4, 199] = float("nan")
        w = torch.ones(200, device="cuda", dtype=dtype)
        q, scale, _ = dion.rmsnorm_int8(x, w, eps=0.01)
        assert scale[1] == 0 and not q[1].any()
        assert torch.isnan(scale[3]) and torch.isnan(scale[4]) and not q[3:5].any()
        clean = dion.rmsnorm_int8(x[[0, 2, 5]], w, eps=0.01)
        assert torch.equal(q[[0, 2, 5]], clean[0]) and torch.equal(scale[[0, 2, 5]], clean[1])
        y, _, rstd = dion.rmsnorm(x, w, eps=0.01)
        assert not y[1].any() and torch.isnan(y[4]).all()
        ref, _ = O.rmsnorm(n64(x[2:3]), np.ones(200), 0.01)
        within(y[2:3], ref, (U[dtype] + ACC) * np.abs(ref) + 1e-38, "tiny row")
        # quantised as they are
        q, scale = dion.int8_quantize(x * 1e-20 * 1e-20 if dtype == torch.float32 else x)
        assert scale[1] == 0 and not q[1].any() and torch.isnan(scale[3]) and torch.isnan(scale[4])
        if dtype == torch.float32:
            assert (scale[[0, 2, 5]] == 0).all() and not q[[0, 2, 5]].any()   # below 2^-119


@pytest.mark.parametrize("rows,cols", [(0, 8), (1, 1), (3, 5), (40, 129), (7, 4096), (2, 30000), (300, 64)])
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("fp16", 3), ("fp32", 4)])
def test_quantize_codes_are_the_definition(dion, rows, cols, dtype, pad):
    """Elementwise fp32 with correctly rounded division (here: in float64, then rounded): equal bit for bit."""
    x = strided(randn(21, (rows, cols), DT[dtype], 5.0), pad if rows else 0, 1)
    q, scale = dion.int8_quantize(x)
    a = x.float().abs().amax(1)
    assert torch.equal(scale, (a.double() / 127).float())
    assert torch.equal(q.float(), torch.round(x.float() * (127 * (1 / a.double()).float())[:, None]))
    for out in (torch.bfloat16, torch.float16, torch.float32):
        assert torch.equal(dion.int8_dequantize(q, scale, out), (q.float() * scale[:, None]).to(out))


# ------------------------------------------------------------- 8-bit products
LINEAR = [(1, 1, 1), (1, 5, 0), (2, 3, 17), (1, 64, 64), (1, 1000, 333), (3, 257, 128), (5, 31, 4096), (16, 96, 640),
          (17, 100, 300), (24, 520, 1024), (33, 129, 65), (64, 256, 2048), (65, 300, 511), (100, 64, 14336),
          (128, 128, 128), (129, 257, 200), (200, 1000, 777), (256, 512, 1024), (300, 270, 130), (515, 777, 640),
          (1030, 260, 384), (70, 90, 48), (300, 140, 208), (1500, 1300, 1040), (4100, 4200, 400)]


@pytest.mark.parametrize("m,n,k", LINEAR)
@pytest.mark.parametrize("out,bias,pad", [("bf16", None, 0), ("fp32", "fp32", 5), ("fp16", "bf16", 16)])
def test_int8_linear(dion, m, n, k, out, bias, pad):
    g = torch.Generator(device="cuda")
    g.manual_seed(m * 7 + n * 3 + k)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda").to(torch.int8)
    b = torch.randint(-128, 128, (n, k), generator=g, device="cuda").to(torch.int8)
    sa = 0.001 + torch.rand(m, generator=g, device="cuda") * 0.01
    sb = (0.001 + torch.rand(n, generator=g, device="cuda")) * 0.02
    bv = None if bias is None else torch.randn(n, generator=g, device="cuda").to(DT[bias])
    if k:
        a, b = strided(a, pad, pad // 2), strided(b, pad, pad // 3)
    y = dion.int8_linear(a, sa, b, sb, bias=bv, out_dtype=DT[out])
    assert y.shape == (m, n) and y.dtype == DT[out]
    prod = O.int8_linear(n64(a), n64(sa), n64(b), n64(sb))
    bb = 0 if bias is None else n64(bv)
    tol = U[DT[out]] * np.abs(prod + bb) + 2.0 ** -22 * (np.abs(prod) + np.abs(bb)) + TINY[DT[out]]
    within(y, prod + bb, tol, "out")


def test_int8_linear_extremes(dion):
    """The longest sum of the largest products stays inside 32 bits; a NaN scale shows in its row alone."""
    k = (1 << 17) - 1
    a = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    b = torch.full((5, k), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    one = torch.ones(5, device="cuda")
    sa = torch.tensor([1.0, float("nan"), 2.0], device="cuda")
    y = dion.int8_linear(a, sa, b, one, out_dtype=torch.float32)
    assert torch.isnan(y[1]).all()
    want = torch.tensor([16384.0 * k, -16256.0 * k, 16384.0 * k, 16384.0 * k, 16384.0 * k], dtype=torch.float64)
    assert torch.equal(y[0].cpu(), want.float()) and torch.equal(y[2].cpu(), (2 * want).float())


@pytest.mark.parametrize("m,n", [(1, 37), (5, 300), (16, 21), (3, 14001), (40, 70)])
@pytest.mark.parametrize("k,gap", [(5, 2), (127, 0), (130, 3), (131, 0), (133, 0), (128, 1), (132, 5), (2051, 0), (2048, 7),
                                   (14339, 0)])
@pytest.mark.parametrize("start", [0, 1, 4])
def test_int8_linear_rows_inside_dwords(dion, m, n, k, gap, start):
    """Rows at any byte, between other bytes that must not count: with scales of one the output is the exact sum,
    rounded once."""
    def matrix(rows, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        whole = torch.full((start + rows * (k + gap),), -128, dtype=torch.int8, device="cuda")
        v = whole[start:].view(rows, k + gap)[:, :k]
        v.copy_(torch.randint(-128, 128, (rows, k), generator=g, device="cuda"))
        return v
    a, b = matrix(m, k), matrix(n, k + 1)
    one = torch.ones(max(m, n), device="cuda")
    y = dion.int8_linear(a, one[:m], b, one[:n], out_dtype=torch.float32)
    assert torch.equal(y, (a.double() @ b.double().t()).float())


def test_int8_linear_leading_dimensions_and_order(dion):
    """Tokens with leading dimensions; every row is computed as it is alone."""
    a = torch.randint(-127, 128, (4, 10, 192), device="cuda").to(torch.int8)
    b = torch.randint(-127, 128, (70, 192), device="cuda").to(torch.int8)
    sa, sb = torch.rand(4, 10, device="cuda"), torch.rand(70, device="cuda")
    y = dion.int8_linear(a, sa, b, sb, out_dtype=torch.float32)
    assert y.shape == (4, 10, 70)
    for i, j in ((0, 0), (3, 9), (1, 5)):
        assert torch.equal(dion.int8_linear(a[i, j:j + 1], sa[i, j:j + 1], b, sb, out_dtype=torch.float32)[0], y[i, j])


# ---------------------------------------------------------------- distillation
def distill_case(rows, vocab, k, dt, tdt, seed=0, spread=2.0, idx_dtype=torch.int64):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + rows * 31 + vocab)
    z = (torch.randn((rows, vocab), generator=g, device="cuda") * spread).to(dt)
    t = (torch.randn((rows, k), generator=g, device="cuda") * 3).to(tdt)
    idx = torch.randint(vocab, (rows, k), generator=g, device="cuda")   # repeated ones among them
    idx[torch.rand((rows, k), generator=g, device="cuda") < 0.1] = -1
    return z, t, idx.to(idx_dtype)


def distill_check(dion, z, t, idx, temp, gl, pad=0):
    """All three entry points against the oracle; z may be a view with a row stride."""
    dt = z.dtype
    Z, T, I = n64(z), n64(t), idx.cpu().numpy()
    safe = np.where(np.isnan(Z) | (Z == np.inf), 0, Z)   # only in rows that give zeros
    with np.errstate(all="ignore"):
        loss, dz, live = O.distill(safe, T, I, temp)
        m = safe.max(1, keepdims=True)
        u = (safe - m) / temp
        ls = np.log(np.exp(u).sum(1, keepdims=True))
        q = np.exp(u - ls)
    inside = (I >= 0) & (I < Z.shape[1]) & (T != -np.inf)
    ui = np.abs(np.take_along_axis(u, np.where(inside, I, 0), 1)) if I.shape[1] else np.zeros((len(Z), 1))
    tt = np.where(inside, T, -np.inf)
    top = tt.max(1, keepdims=True, initial=-np.inf)
    dt_ = np.where(inside, np.abs(T - np.where(np.isfinite(top), top, 0)) / temp, 0) if I.shape[1] else ui * 0
    dt_ = np.where(dt_ < 120, dt_, 0)   # beyond it p is 0 in fp32 and below 1e-45 in truth
    depth = np.where(inside, ui, 0).max(1, initial=0) + dt_.max(1, initial=0) + np.abs(ls[:, 0]) + 4
    got, stats = dion.distill_topk(z, t, idx, temperature=temp)
    tol = temp ** 2 * (ACC + 2.0 ** -21 * depth)
    within(got, loss, tol, "loss")
    assert not n64(got)[~live].any()
    g = np.ones(len(Z)) if gl is None else n64(gl)
    ref = dz * g[:, None]
    P = np.abs(q * temp - dz) / temp
    with np.errstate(all="ignore"):
        far = np.where(np.isfinite(u), np.abs(u), 0) + np.abs(ls)
    dtol = U[dt] * np.abs(ref) + np.abs(g)[:, None] * temp * (q * (ACC + 2.0 ** -21 * far) + 2.0 ** -20 * P
                                                             + P * 2.0 ** -21 * dt_.max(1, initial=0)[:, None])
    d = dion.distill_topk_backward(gl, z, stats, t, idx, temperature=temp)
    assert d.shape == z.shape and d.dtype == dt
    within(d, ref, dtol + TINY[dt], "dlogits")
    dead = ~live | (g == 0)
    assert not n64(d)[dead].any()
    loss2, d2 = dion.distill_topk_step(z, t, idx, gl, temperature=temp)
    within(loss2, loss, tol, "loss of the step")
    within(d2, ref, dtol + TINY[dt], "dlogits of the step")
    assert not n64(d2)[dead].any()
    # in place
    copy = strided(z.clone(), pad, pad // 2)
    loss3, d3 = dion.distill_topk_step(copy, t, idx, gl, temperature=temp, out=copy)
    assert d3 is copy and torch.equal(d3, d2) and torch.equal(loss3, loss2)
    copy = strided(z.clone(), pad, pad // 2)
    d4 = dion.distill_topk_backward(gl, copy, stats, t, idx, temperature=temp, out=copy)
    assert torch.equal(d4, d)
    return got, d


DISTILL = [(1, 1, 1), (2, 3, 2), (1, 17, 5), (5, 1000, 1), (3, 1023, 64), (16, 4096, 100), (2, 50257, 32),
           (1, 131072, 256), (7, 32001, 17), (300, 257, 8), (40, 8192, 1024),
           (131, 70001, 20), (129, 140000, 5), (600, 20000, 40), (2100, 300, 33), (1100, 9000, 3)]


@pytest.mark.parametrize("rows,vocab,k", DISTILL)
@pytest.mark.parametrize("dtype,tdtype,temp,pad,itype", [("bf16", "bf16", 1.0, 0, torch.int64),
                                                         ("fp32", "fp32", 2.0, 7, torch.int32),
                                                         ("fp16", "fp32", 0.5, 16, torch.int64)])
def test_distill(dion, rows, vocab, k, dtype, tdtype, temp, pad, itype):
    z, t, idx = distill_case(rows, vocab, k, DT[dtype], DT[tdtype], idx_dtype=itype)
    gl = randn(9, (rows,), torch.float32)
    if rows > 4:
        idx[3] = -1
        gl[1] = 0
    distill_check(dion, strided(z, pad, pad // 2), t, idx, temp, gl, pad)


def test_distill_no_teacher_entries(dion):
    z = randn(1, (3, 100), torch.bfloat16)
    t = torch.empty((3, 0), device="cuda")
    loss, d = dion.distill_topk_step(z, t, torch.empty((3, 0), dtype=torch.int64, device="cuda"))
    assert not loss.any() and not d.any()
    z = torch.empty((0, 100), device="cuda")
    loss, d = dion.distill_topk_step(z, torch.empty((0, 4), device="cuda"),
                                     torch.empty((0, 4), dtype=torch.int64, device="cuda"))
    assert loss.shape == (0,) and d.shape == (0, 100)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,copies", [(200, 1), (40000, 1), (200, 30), (40000, 14)])
def test_distill_masked_places(dion, dtype, vocab, copies):
    """-inf and the type's lowest value among the logits of both sides, NaN and
    infinities in rows without a teacher or gradient, indices out of range."""
    dt = DT[dtype]
    z, t, idx = distill_case(10, vocab, 6, dt, dt)
    idx = torch.stack([torch.randperm(vocab, device="cuda")[:6] for _ in range(10)])
    lowest = torch.finfo(dt).min
    hidden = [i for i in range(vocab - 30, vocab)]
    z[0, hidden] = float("-inf")       # a masked part of the vocabulary
    z[1, hidden] = lowest
    idx[0] = torch.arange(6, device="cuda")
    idx[1] = torch.arange(6, device="cuda")
    t[2, 1:] = float("-inf")           # one entry left
    t[3, 2:] = lowest
    t[4] = lowest                      # equal, however low
    idx[5] = torch.tensor([-1, vocab, vocab + 5, -7, 2 ** 40, -2 ** 40], device="cuda")   # none inside
    z[5] = float("nan")
    t[6] = float("-inf")               # none present
    z[6] = float("inf")
    z[7] = float("nan")
    gl = torch.rand(10, device="cuda") + 0.5
    gl[7] = 0                          # no gradient wanted; the loss is NaN
    loss, stats = dion.distill_topk(z, t, idx)
    assert torch.isnan(loss[7])
    # a masked student entry that the teacher wants: infinitely wrong
    z2 = z[:1].clone()
    z2[0, 3] = float("-inf")
    l2, _ = dion.distill_topk(z2, t[:1], idx[:1])
    assert torch.isinf(l2).all()
    t2 = t[:1].clone()
    t2[0, 3] = float("-inf")           # ... and one that it does not
    assert torch.isfinite(dion.distill_topk(z2, t2, idx[:1])[0]).all()
    d = dion.distill_topk_backward(gl, z, stats, t, idx)
    assert not d[5:8].any() and not d[0, hidden].any() and not d[1, hidden].any()
    z[7] = 0
    z[8] = lowest                      # a student with nothing but masks, all equal
    z[9, 5:] = float("-inf")           # almost nothing left of the student
    idx[9] = torch.tensor([0, 1, 2, 3, 4, -1], device="cuda")
    z, t, idx, gl = (v.repeat(copies, *[1] * (v.dim() - 1)) for v in (z, t, idx, gl))
    distill_check(dion, z, t, idx, 0.7, gl)


def test_distill_gradient_against_differences(dion):
    """Directional central differences of the fp32 loss: with a direction of
    norm 1 and step e = 2^-5 the truncation is below e^2 / 6 (third derivatives
    of a log-sum-exp are below one), and a loss of about 8 rounds to 2^-21
    (4e-6 with the sums' errors), over 2e below 1e-4: 4e-4 in all."""
    rows, vocab, e = 2, 300, 2.0 ** -5
    z, t, idx = distill_case(rows, vocab, 9, torch.float32, torch.float32)
    v = randn(33, (rows, vocab), torch.float32)
    v = v / v.norm()
    _, d = dion.distill_topk_step(z, t, idx)
    f = lambda a: float(dion.distill_topk(a, t, idx)[0].double().sum())
    assert abs((f(z + e * v) - f(z - e * v)) / (2 * e) - float((d * v).double().sum())) <= 4e-4


def test_distill_three_dimensions_and_teacher_views(dion):
    z = randn(2, (2, 5, 400), torch.bfloat16)
    full = randn(3, (2, 5, 400), torch.float32)
    t, idx = full.topk(12, dim=-1)
    loss, d = dion.distill_topk_step(z, t[..., :7], idx[..., :7])
    assert loss.shape == (2, 5) and d.shape == z.shape
    flat, df = dion.distill_topk_step(z.view(10, 400), t[..., :7].reshape(10, 7), idx[..., :7].reshape(10, 7))
    assert torch.equal(loss.view(-1), flat) and torch.equal(d.reshape(10, 400), df)


# ------------------------------------------------------- the operators in use
def test_autograd_functions(dion):
    """rms_norm and distill_loss under torch's automatic differentiation against the same in float64."""
    rows, cols, vocab, k = 6, 80, 500, 9
    x = randn(1, (rows, cols), torch.float32).requires_grad_()
    r = randn(2, (rows, cols), torch.float32).requires_grad_()
    w = (1 + 0.1 * randn(3, (cols,), torch.float32)).requires_grad_()
    head = (randn(4, (vocab, cols), torch.float32) / 8).requires_grad_()
    t, idx = randn(5, (rows, vocab), torch.float32, 2.0).topk(k)
    y, h = dion.rms_norm(x, w, r)
    loss = dion.distill_loss(y @ head.t(), t, idx, 1.5).mean() + (h * h).mean()
    loss.backward()
    X, R, W, H = (v.detach().double().cpu().requires_grad_() for v in (x, r, w, head))
    s = X + R
    Y = s * torch.rsqrt(s.pow(2).mean(1, keepdim=True) + 1e-6) * W
    p = torch.softmax(t.double().cpu() / 1.5, 1)
    logq = torch.log_softmax(Y @ H.t() / 1.5, 1).gather(1, idx.cpu())
    want = 1.5 ** 2 * (p * (p.log() - logq)).sum(1).mean() + (s * s).mean()
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-5 * abs(float(want.detach()))
    # fp32 products of 80 and 500 terms in between: 1e-4 of each gradient's size
    for a, b in ((x, X), (r, R), (w, W), (head, H)):
        assert float((a.grad.double().cpu() - b.grad).norm()) <= 1e-4 * float(b.grad.norm())


def test_streams_and_graphs(dion):
    """On a stream of its own, and captured into a graph that is replayed on new inputs."""
    z, t, idx = distill_case(9, 3000, 8, torch.bfloat16, torch.float32)
    x, w = randn(1, (9, 256), torch.bfloat16), torch.ones(256, device="cuda", dtype=torch.bfloat16)
    r = randn(2, (9, 256), torch.bfloat16)
    b, sb = dion.int8_quantize(randn(3, (100, 256), torch.bfloat16))

    def work(stream=None):
        q, scale, h = dion.rmsnorm_int8(x, w, residual=r, stream=stream)
        y = dion.int8_linear(q, scale, b, sb, stream=stream)
        n, hh, rstd = dion.rmsnorm(x, w, residual=r, stream=stream)
        dx, dw = dion.rmsnorm_backward(n, hh, w, rstd, stream=stream)
        loss, d = dion.distill_topk_step(z, t, idx, stream=stream)
        return y, h, dx, dw, loss, d

    want = [v.clone() for v in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = work(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(got, want):
        assert torch.equal(a, c)
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        z.copy_(randn(50 + i, tuple(z.shape), torch.bfloat16, 2.0))
        x.copy_(randn(60 + i, tuple(x.shape), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        for a, c in zip(got, work()):
            assert torch.equal(a, c), i
        torch.cuda.synchronize()


def test_outputs_write_nothing_beside(dion):
    """Guard values around every output that the caller owns stay as they are."""
    z, t, idx = distill_case(5, 1001, 6, torch.bfloat16, torch.float32)
    wide = torch.full((7, 1030), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[1:6, 11:1012]
    dion.distill_topk_step(z, t, idx, out=out)
    assert torch.equal(out, dion.distill_topk_step(z, t, idx)[1])
    wide[1:6, 11:1012] = 3.0
    assert (wide == 3.0).all()


def test_profile_records(dion):
    x, w = randn(1, (4, 64), torch.bfloat16), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    dion.profile_enable(True)
    try:
        q, s, _ = dion.rmsnorm_int8(x, w)
        dion.int8_linear(q, s, q, s)
        names = [r[0] for r in dion.profile_records()]
    finally:
        dion.profile_enable(False)
    assert names == ["rmsnorm_int8", "int8_linear"]


# ------------------------------------------------------------------- refusals
def test_refusals(dion):
    E = dion.DionError
    x = randn(1, (4, 32), torch.bfloat16)
    w = torch.ones(32, device="cuda", dtype=torch.bfloat16)
    q, s = dion.int8_quantize(x)
    z, t, idx = distill_case(4, 50, 3, torch.bfloat16, torch.float32)
    stats = torch.zeros(4, 2, device="cuda")
    bad = [
        lambda: dion.rmsnorm(x.cpu(), w),
        lambda: dion.rmsnorm(x.double(), w),
        lambda: dion.rmsnorm(x.t(), w),
        lambda: dion.rmsnorm(x, w[:31]),
        lambda: dion.rmsnorm(x, w.half()),
        lambda: dion.rmsnorm(x, w, residual=x[:3]),
        lambda: dion.rmsnorm(x, w, residual=x.float()),
        lambda: dion.rmsnorm(x, w, eps=-1.0),
        lambda: dion.rmsnorm(x, w, eps=float("nan")),
        lambda: dion.rmsnorm(x[:, :0], w[:0]),
        lambda: dion.rmsnorm(x[:1].expand(4, 32), w),
        lambda: dion.rmsnorm(torch.zeros((1, 65537), device="cuda"), torch.ones(65537, device="cuda")),
        lambda: dion.rmsnorm_backward(x, x, w, torch.ones(3, device="cuda")),
        lambda: dion.rmsnorm_backward(x.float(), x, w, torch.ones(4, device="cuda")),
        lambda: dion.rmsnorm_backward(x, x, w, torch.ones(4, device="cuda"),
                                      workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: dion.int8_quantize(q),
        lambda: dion.int8_dequantize(x, s),
        lambda: dion.int8_dequantize(q, s, torch.int8),
        lambda: dion.int8_linear(x, s, q, s),
        lambda: dion.int8_linear(q, s, q[:, :16], s),
        lambda: dion.int8_linear(q, s[:3], q, s),
        lambda: dion.int8_linear(q, s, q, s.half()),
        lambda: dion.int8_linear(q, s, q, s, bias=torch.ones(3, device="cuda")),
        lambda: dion.int8_linear(q, s, q, s, out_dtype=torch.int32),
        lambda: dion.int8_linear(torch.zeros((1, 1 << 17), dtype=torch.int8, device="cuda"), s[:1],
                                 torch.zeros((1, 1 << 17), dtype=torch.int8, device="cuda"), s[:1]),
        lambda: dion.distill_topk(z, t[:3], idx[:3]),
        lambda: dion.distill_topk(z, t, idx[:, :2]),
        lambda: dion.distill_topk(z, t, idx.float()),
        lambda: dion.distill_topk(z, t, idx, temperature=0.0),
        lambda: dion.distill_topk(z, t, idx, temperature=float("inf")),
        lambda: dion.distill_topk(z.t(), t, idx),
        lambda: dion.distill_topk(z, torch.zeros((4, 1025), device="cuda"),
                                  torch.zeros((4, 1025), dtype=torch.int64, device="cuda")),
        lambda: dion.distill_topk_step(z, t, idx, grad_loss=torch.ones(3, device="cuda")),
        lambda: dion.distill_topk_step(z, t, idx, out=torch.empty((4, 51), dtype=z.dtype, device="cuda")),
        lambda: dion.distill_topk_backward(None, z, stats[:3], t, idx),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(E):
            f()
            pytest.fail(f"call {i} was not refused")
    # overlapping outputs
    buf = torch.zeros(4 * 50 + 10, dtype=torch.bfloat16, device="cuda")
    a, o = buf[:200].view(4, 50), buf[10:210].view(4, 50)
    with pytest.raises(E):
        dion.distill_topk_step(a, t, idx, out=o)
