"""Calls of the training-step operators at the edges of their plans, on the GPU: the smallest uses of scratch, masks
anywhere in a row, teacher tensors that are views on other streams, the longest and the emptiest shapes.

Tolerances are those of the operators' other tests: u is the largest relative rounding error of the output's type, and
an fp32 sum is allowed ACC = 2^-15 of its magnitudes' sum.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import train_oracle as O  # noqa: E402
from test_gpu_train_ops import distill_case, distill_check  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ACC = 2.0 ** -15


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


def n64(t):
    return t.detach().double().cpu().numpy()


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(seed, shape):
    return torch.randint(-128, 128, shape, generator=generator(seed), device="cuda").to(torch.int8)


# ------------------------------------------------------------- 8-bit products
@pytest.mark.parametrize("m,n,k,start", [(1, 1, 7168, 0), (1, 32, 7168, 0), (2, 16, 7168, 0), (16, 2, 7168, 0),
                                         (1, 8, 14336, 0), (1, 16, 14336, 0), (17, 1, 128, 3), (32, 4, 64, 1)])
def test_int8_linear_with_little_scratch(dion, m, n, k, start):
    """The sums of the splits, or the aligned copy of b, take 256 bytes at most.  With scales of one the output is the
    exact sum, rounded once."""
    a = codes(m, (m, k))
    b = codes(n + 100, (start + n * k,))[start:].view(n, k)
    one = torch.ones(max(m, n), device="cuda")
    y = dion.int8_linear(a, one[:m], b, one[:n], out_dtype=torch.float32)
    assert torch.equal(y, (a.double() @ b.double().t()).float())


@pytest.mark.parametrize("m,n,k", [(70000, 64, 14336), (70001, 3, 8192)])
def test_int8_linear_joins_the_splits_of_many_tokens(dion, m, n, k):
    """More tokens than a grid has rows of blocks, k in splits."""
    a, b = codes(1, (m, k)), codes(2, (n, k))
    one = torch.ones(m, device="cuda")
    y = dion.int8_linear(a, one, b, one[:n], out_dtype=torch.float32)
    for rows in (slice(0, 100), slice(32700, 32800), slice(65500, 65600), slice(m - 100, m)):
        assert torch.equal(y[rows], (a[rows].double() @ b.double().t()).float())


@pytest.mark.parametrize("cols", [(1 << 28) + 5, (1 << 31) - 1])
def test_dequantize_the_longest_rows(dion, cols):
    """More blocks than a grid has along one dimension, and the last elements that 32-bit indexes reach."""
    q = codes(3, (1, cols))
    y = dion.int8_dequantize(q, torch.full((1,), 0.5, device="cuda"))
    for lo in (0, (1 << 27) - 50, (1 << 28) - 50, cols // 2, cols - 5000):
        assert torch.equal(y[0, lo:lo + 5000].float(), q[0, lo:lo + 5000].float() * 0.5)


@pytest.mark.parametrize("lead", [(2, 3), (6,), (2, 0), (), (1, 2, 3)])
def test_int8_linear_of_nothing(dion, lead):
    """k = 0: every token's row is the bias, with leading dimensions too."""
    n = 5
    bias = torch.randn(n, device="cuda")
    a, b = (torch.zeros(s, dtype=torch.int8, device="cuda") for s in ((*lead, 0), (n, 0)))
    y = dion.int8_linear(a, torch.ones(lead, device="cuda"), b, torch.ones(n, device="cuda"), bias=bias,
                         out_dtype=torch.float32)
    assert y.shape == (*lead, n) and torch.equal(y, bias.expand(*lead, n))


def test_int8_linear_copies_operands_of_any_size(dion):
    """An unaligned operand of more than 2^32 pieces of 16 bytes (64 GiB)."""
    m, k = 1 << 22, 16385
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB of free GPU memory")
    a = torch.zeros((m, k), dtype=torch.int8, device="cuda")
    rows = [0, 1, 12345, m // 2, m - 2, m - 1]
    a[rows] = codes(5, (len(rows), k))
    b = codes(6, (1, k))
    y = dion.int8_linear(a, torch.ones(m, device="cuda"), b, torch.ones(1, device="cuda"), out_dtype=torch.float32)[:, 0]
    want = torch.zeros(m, device="cuda")
    want[rows] = (a[rows].double() @ b.double().t()).float()[:, 0]
    assert torch.equal(y, want)
    del a, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("k", [64, 500, 4096])
@pytest.mark.parametrize("bias", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
def test_int8_linear_of_a_token_does_not_depend_on_the_others(dion, k, bias, out):
    """Every kernel rounds alike: the sum, its product with each scale, the bias' addition, the output."""
    n = 300
    a, b = codes(1, (600, k)), codes(2, (n, k))
    sa, sb = (torch.rand(s, generator=generator(s), device="cuda") for s in (600, n))
    v = None if bias is None else (torch.randn(n, generator=generator(3), device="cuda") * 1000).to(bias)
    if out == torch.float16:
        sb = sb * 1e-3   # inside its range
    want = (a.double() @ b.double().t()).float() * sa[:, None] * sb
    want = (want if v is None else want + v.float()).to(out)
    for m in (1, 5, 16, 17, 40, 129, 600):
        assert torch.equal(dion.int8_linear(a[:m], sa[:m], b, sb, bias=v, out_dtype=out), want[:m])


# ---------------------------------------------------------------- distillation
@pytest.mark.parametrize("rows,vocab,k,dt", [(1, 128256, 32, torch.bfloat16), (2, 128256, 1, torch.float16),
                                             (1, 70001, 8, torch.float32), (1, 90000, 4, torch.float32)])
def test_distill_with_little_scratch(dion, rows, vocab, k, dt):
    """The parts of the shared rows take 256 bytes at most."""
    z, t, idx = distill_case(rows, vocab, k, dt, torch.float32)
    idx[0, 0] = 5
    distill_check(dion, z, t, idx, 1.5, torch.rand(rows, device="cuda") + 0.5)


# one vocabulary for each way of holding a row, and one too long to hold
MASKED = [(1001, 6, torch.bfloat16), (17001, 6, torch.bfloat16), (30000, 6, torch.float16), (60000, 6, torch.bfloat16),
          (90000, 130, torch.bfloat16), (140001, 130, torch.bfloat16), (9000, 6, torch.float32),
          (20001, 6, torch.float32), (31000, 6, torch.float32), (50000, 130, torch.float32)]


@pytest.mark.parametrize("vocab,rows,dt", MASKED)
@pytest.mark.parametrize("mask", ["lowest", -1e30, -1e20, -1e9, "-inf"])
@pytest.mark.parametrize("temp", [0.5, 1.0, 4.0])
def test_distill_masks_anywhere(dion, vocab, rows, dt, mask, temp):
    """Masked runs at the front, in the middle, in every other 16 bytes, and everywhere but at the end of a row.  Their
    exponentials are exactly 0 beside ordinary logits, in 64 bits as in 32."""
    value = {"lowest": torch.finfo(dt).min, "-inf": float("-inf")}.get(mask, mask)
    if isinstance(value, float) and value < torch.finfo(dt).min and mask != "-inf":
        value = torch.finfo(dt).min
    z, t, _ = distill_case(rows, vocab, 5, dt, torch.float32, seed=3)
    chunk = 16 // z.element_size()
    at = torch.arange(vocab, device="cuda")
    hidden = [at < chunk, at < vocab // 2, (at >= vocab // 3) & (at < vocab // 3 + 40 * chunk), (at // chunk) % 2 == 0,
              at < vocab - 7, (at >= chunk) & (at < vocab - chunk)]
    idx = torch.empty((rows, 5), dtype=torch.int64, device="cuda")
    for r in range(rows):
        if r < 6 or r >= rows - 6:   # the rows between stay as they are
            z[r, hidden[r % 6]] = value
            idx[r] = at[~hidden[r % 6]][-5:]
        else:
            idx[r] = torch.randperm(vocab, device="cuda")[:5]
    loss, d = distill_check(dion, z, t, idx, temp, torch.rand(rows, device="cuda") + 0.5)
    assert torch.isfinite(loss).all() and torch.isfinite(d.float()).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_distill_far_from_zero(dion, dt):
    """A row's logits around a large value of either sign, so that the reference is on one side of 2^20 or the other:
    they are exact in the type, and only their differences count."""
    step = 4096.0 if dt == torch.bfloat16 else 1.0
    base = torch.tensor([0.0, 2.0 ** 19, -2.0 ** 19, 2.0 ** 20 - 2 * step, 2.0 ** 20 + 2 * step, -2.0 ** 20 + 2 * step,
                         -2.0 ** 20 - 2 * step, 2.0 ** 22], device="cuda")
    vocab, k, temp = 9001, 6, 3.0 * step
    steps = torch.randint(-3, 4, (8, vocab), generator=generator(5), device="cuda").float()
    z = (base[:, None] + steps * step).to(dt)
    assert torch.equal(z.float(), base[:, None] + steps * step) or dt == torch.bfloat16
    t, idx = z.float().topk(k)
    # D of the tolerance is a few units for all rows: the exponents are within 2 of one another
    Z, T, I = n64(z), n64(t), idx.cpu().numpy()
    ref, dz, _ = O.distill(Z, T, I, temp)
    tol = temp ** 2 * (ACC + 2.0 ** -21 * 16)
    loss, stats = dion.distill_topk(z, t, idx, temperature=temp)
    step_loss, d = dion.distill_topk_step(z, t, idx, temperature=temp)
    back = dion.distill_topk_backward(None, z, stats, t, idx, temperature=temp)
    q = np.exp((Z - Z.max(1, keepdims=True)) / temp)
    q /= q.sum(1, keepdims=True)
    P = np.abs(q * temp - dz) / temp
    dtol = U[dt] * np.abs(dz) + temp * (q * (ACC + 2.0 ** -21 * 16) + 2.0 ** -20 * P + 2.0 ** -21 * 4 * P)
    for got, want, by in ((loss, ref, tol), (step_loss, ref, tol), (d, dz, dtol), (back, dz, dtol)):
        assert (np.abs(n64(got) - want) <= by).all()


@pytest.mark.parametrize("rows,vocab,k,temp,dt", [(1021, 32001, 100, 1.5, torch.float32), (700, 1499, 43, 1.0, torch.float16),
                                                  (2000, 1461, 5, 0.5, torch.bfloat16), (900, 2449, 253, 1.0, torch.float32),
                                                  (500, 50257, 64, 2.0, torch.bfloat16)])
def test_distill_is_as_exact_as_elementary_operations_in_fp32(dion, rows, vocab, k, temp, dt):
    """The error against 64 bits over all rows (2-norm) of the loss, and of an fp32 gradient, is no larger than 1.5 times
    that of the formula in torch's fp32 operations, which round every step once: the kernels round no more often."""
    g = generator(7)
    z = torch.randn((rows, vocab), generator=g, device="cuda") * 2
    idx = torch.rand((rows, vocab), generator=g, device="cuda").topk(k).indices
    t = 14 - torch.rand((rows, k), generator=g, device="cuda").mul(1.2 * 12 / k).cumsum(1)
    z.scatter_(1, idx, t - 3 + torch.randn((rows, k), generator=g, device="cuda"))
    z = z.to(dt)

    def formula(z, t):
        u, v = (t - t.amax(1, keepdim=True)) / temp, (z - z.amax(1, keepdim=True)) / temp
        p, logs = torch.softmax(u, 1), torch.log(torch.exp(v).sum(1, keepdim=True))
        logp = u - torch.log(torch.exp(u).sum(1, keepdim=True))
        loss = temp ** 2 * (p * (logp - (v.gather(1, idx) - logs))).sum(1)
        return loss, temp * torch.exp(v - logs).scatter_add_(1, idx, -p)

    exact, plain = formula(z.double(), t.double()), formula(z.float(), t)
    loss, stats = dion.distill_topk(z, t, idx, temperature=temp)
    step = dion.distill_topk_step(z, t, idx, temperature=temp)
    got = [(loss, 0), (step[0], 0)]
    if dt == torch.float32:
        got += [(step[1], 1), (dion.distill_topk_backward(None, z, stats, t, idx, temperature=temp), 1)]
    for value, i in got:
        far = float((value.double() - exact[i]).norm())
        assert far <= 1.5 * float((plain[i].double() - exact[i]).norm()), (i, far)


def test_distill_teacher_views_on_another_stream(dion):
    """Teacher tensors that are slices are copied on the stream that reads them: the call orders itself after nothing
    that the caller's own stream still has before it."""
    rows, vocab, k = 64, 5000, 7
    z, t, idx = distill_case(rows, vocab, 2 * k, torch.bfloat16, torch.float32)
    tc, ic = t[:, :k].contiguous(), idx[:, :k].contiguous()
    stats = dion.distill_topk(z, tc, ic)[1]
    busy = torch.randn(8192, 8192, device="cuda")
    side = torch.cuda.Stream()
    calls = (lambda t, i, s: dion.distill_topk_step(z, t, i, stream=s),
             lambda t, i, s: (*dion.distill_topk(z, t, i, stream=s),
                              dion.distill_topk_backward(None, z, stats, t, i, stream=s)))
    for call in calls:
        want = call(tc, ic, None)
        torch.cuda.synchronize()   # the inputs are there for every stream
        for _ in range(20):   # 20 ms and more on the current stream
            busy = busy @ busy * 1e-3
        got = call(t[:, :k], idx[:, :k], side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------- automatic differentiation
def test_second_derivatives_are_refused(dion):
    """A penalty on a gradient beside another path: it must not train without the penalty, silently."""
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    r = torch.randn(4, 64, device="cuda", requires_grad=True)
    t, idx = torch.randn(4, 64, device="cuda").topk(5)
    for f in (lambda: dion.distill_loss(x, t, idx).sum(), lambda: dion.rms_norm(x, w).pow(2).sum(),
              lambda: sum(v.pow(2).sum() for v in dion.rms_norm(x, w, r))):
        loss = f() + (x ** 3).sum()
        grad, = torch.autograd.grad(loss, x, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiate twice"):
            (loss + grad.pow(2).sum()).backward()
        f().backward()   # once is as before


def test_autograd_functions_take_any_strides(dion):
    """Transposed, permuted, expanded and sliced activations give what their contiguous copies give, gradients included."""
    base = torch.randn(6, 10, 64, device="cuda")
    w = torch.randn(128, device="cuda")[::2]
    views = [lambda b: b[0, :, :].t(), lambda b: b.permute(1, 0, 2), lambda b: b[:, :1, :].expand(6, 10, 64),
             lambda b: b[..., ::2], lambda b: b[:, 3, :40], lambda b: b]
    for view in views:
        t, idx = torch.randn(view(base).shape, device="cuda").topk(3)
        for f in (lambda x, w: dion.rms_norm(x, w).pow(2).sum(),
                  lambda x, w: sum(v.pow(2).sum() for v in dion.rms_norm(x, w, (x * 0.5).contiguous())),
                  lambda x, w: sum(v.pow(2).sum() for v in dion.rms_norm(x.contiguous(), w, x)),
                  lambda x, w: dion.distill_loss(x, t, idx, 2.0).sum()):
            got = []
            for dense in (False, True):
                b, v = base.clone().requires_grad_(), w[:view(base).shape[-1]]
                v = v if v.numel() == view(base).shape[-1] else torch.ones(view(base).shape[-1], device="cuda")
                x = view(b)
                y = f(x.contiguous() if dense else x, v.contiguous() if dense else v)
                y.backward()
                got.append((y.detach(), b.grad))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_rms_norm_with_an_unused_output(dion, monkeypatch):
    """Either output alone: the other's gradient is absent, not a tensor of zeros that the kernel reads."""
    import orthogonalized_optimizer_step_amd.train_ops as T
    seen, inner = [], T.rmsnorm_backward
    monkeypatch.setattr(T, "rmsnorm_backward", lambda dy, h, w, rstd, dh=None: seen.append(dh is None) or inner(dy, h, w, rstd, dh))
    x, r, w = (torch.randn(s, device="cuda", requires_grad=True) for s in ((5, 48), (5, 48), (48,)))
    g = torch.randn(5, 48, device="cuda")
    dx, dr, dw = torch.autograd.grad(dion.rms_norm(x, w, r)[0], (x, r, w), g)
    _, h, rstd = dion.rmsnorm(x.detach(), w.detach(), residual=r.detach())
    want = inner(g, h, w.detach(), rstd)
    assert seen == [True] and torch.equal(dx, want[0]) and torch.equal(dr, want[0]) and torch.equal(dw, want[1])
    dx, dr, dw = torch.autograd.grad(dion.rms_norm(x, w, r)[1], (x, r, w), g, allow_unused=True)
    assert seen == [True] and torch.equal(dx, g) and torch.equal(dr, g) and dw is None
