"""What the sums of the log probabilities keep: errors against 64 bits beside those of elementary fp32 operations, signs of
log probabilities and entropies, and rows of very many logits."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def peaked(rows, vocab, dtype):
    """Normal logits of spread 2, eight of each row raised by up to 8, one of them the row's token."""
    g = gen(rows + vocab)
    z = torch.randn((rows, vocab), generator=g, device="cuda") * 2
    some = torch.randint(vocab, (rows, 8), generator=g, device="cuda")
    z.scatter_add_(1, some, 8 * torch.rand((rows, 8), generator=g, device="cuda"))
    return z.to(dtype), some[:, 0].contiguous()


def formula(z, t, temp):
    """log of the sum, log probability and entropy, one elementary operation after another in z's precision"""
    u = z / temp
    u = u - u.amax(1, keepdim=True)
    e = torch.exp(u)
    s = e.sum(1, keepdim=True)
    logq = u - torch.log(s)
    return torch.log(s)[:, 0], logq.gather(1, t[:, None])[:, 0], -(e / s * logq).sum(1)


@pytest.mark.parametrize("temp", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("rows,vocab", [(512, 50257), (512, 128256), (64, 128256), (32, 128256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_are_as_exact_as_elementary_operations_in_fp32(dion, rows, vocab, temp, dtype):
    """The root mean square of the errors over 512 rows (of 32 and 64 rows a call) is no larger than 1.25 times that of the
    formula in torch's fp32 operations.  Over 512 rows a root mean square is itself uncertain by 1 / sqrt(1024) = 3 %, so
    that two of them that are equal differ by less than 1.25, eight times that."""
    z, t = peaked(512, vocab, dtype)
    got = [[], [], []]
    for i in range(0, 512, rows):
        lp, ent, stats = dion.token_logprobs(z[i:i + rows], t[i:i + rows], temperature=temp)
        for a, b in zip(got, (stats[:, 3], lp, ent)):
            a.append(b)
    want = [torch.cat(p) for p in zip(*(formula(z[i:i + 64].double(), t[i:i + 64], temp) for i in range(0, 512, 64)))]
    plain = formula(z.float(), t, temp)
    rms = lambda a, b: float((a.double() - b).pow(2).mean().sqrt())
    for what, a, p, w in zip(("log of the sum", "logprob", "entropy"), got, plain, want):
        far, limit = rms(torch.cat(a), w), rms(p, w)
        assert far <= 1.25 * limit, what


@pytest.mark.parametrize("temp", [0.3, 0.5, 0.7, 1.0, 2.0])
@pytest.mark.parametrize("rows,vocab", [(40, 1000), (300, 1000), (300, 50257), (40, 128256), (8, 128256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_signs_of_certain_and_nearly_certain_rows(dion, rows, vocab, temp, dtype):
    """No log probability is above 0 and no entropy below it.  A row with one finite logit (or equal ones alone) has them
    exactly: 0 and 0, whatever the logit."""
    g = gen(rows + vocab)
    z = torch.randn((rows, vocab), generator=g, device="cuda") * 2
    at = torch.randint(vocab, (rows,), generator=g, device="cuda")
    peak = torch.randn((rows,), generator=g, device="cuda") * 12 + 3
    kind = torch.arange(rows, device="cuda") % 4
    z[kind == 0] = -float("inf")               # one finite logit
    z[kind == 1] = torch.finfo(dtype).min      # one above the type's lowest value
    z[kind == 2] -= 60                         # nearly certain
    z[torch.arange(rows, device="cuda"), at] = torch.where(kind == 3, z[torch.arange(rows, device="cuda"), at], peak)
    z = z.to(dtype)
    lp, ent, _ = dion.token_logprobs(z, at, temperature=temp)
    top, index, lp2, ent2 = dion.top_logprobs(z, 5, at, temperature=temp)
    for l, e in ((lp, ent), (lp2, ent2)):
        assert (l <= 0).all() and (e >= 0).all()
        assert not l[kind < 2].any() and not e[kind < 2].any()
    assert (top <= 0).all() and not top[kind < 2, 0].any() and torch.equal(index[kind < 2, 0], at[kind < 2])


@pytest.mark.parametrize("rows,vocab,dtype,far", [
    (257, 1 << 20, torch.bfloat16, 0), (257, (1 << 21) + 5, torch.float32, 0), (40, 1 << 24, torch.bfloat16, 0),
    (2, 1 << 28, torch.bfloat16, 0), (1, (1 << 28) + 4097, torch.float32, 0), (1, 1 << 30, torch.bfloat16, 0),
    (257, (1 << 26) + 9, torch.bfloat16, 0), (40, 1 << 28, torch.bfloat16, 0),
    (257, (1 << 21) + 5, torch.float32, 3e5), (1, (1 << 28) + 4097, torch.float32, 3e5)])   # fp32 numbers, 1/32 apart
def test_sums_of_very_many_equal_terms(dion, rows, vocab, dtype, far):
    """One logit above all others, which are equal: each of their terms rounds the same way wherever sums have the same
    size.  s = 1 + (vocab - 1) exp(-d), entropy log s + (vocab - 1) exp(-d) d / s.  An fp32 sum in which no partial sum runs
    over more than 1024 terms, and a term goes through 1024 additions of at most 2^-24 each, is off by at most 2^-14 of
    itself, and its logarithm by as much; the second sum is off by as much of itself.  (Exponentials: 2^-22 of their own.)"""
    z = torch.full((rows, vocab), far, device="cuda", dtype=dtype)
    t = torch.full((rows,), 3, device="cuda")
    one = torch.ones(rows, device="cuda")
    for d in (i / 16 for i in range(80, 257)):   # numbers of bf16, 16 at most
        z[:, 3] = far + d
        lp, ent, stats = dion.token_logprobs(z, t)
        rest = (vocab - 1) * math.exp(-d)
        s = 1 + rest
        assert float((stats[:, 3].double() - math.log(s)).abs().max()) <= 2.0 ** -14 + 2.0 ** -21 * math.log(s), d
        assert float((lp.double() + math.log(s)).abs().max()) <= 2.0 ** -14 + 2.0 ** -21 * math.log(s), d
        want = math.log(s) + rest * d / s
        assert float((ent.double() - want).abs().max()) <= 2.0 ** -14 * (1 + rest * d / s) + 2.0 ** -20 * want, d
    # their gradient: of the token's logit 1 - 1 / s, which an error of 2^-14 s in s moves by 2^-14 / s; of the others -q
    del lp, ent
    grad = dion.token_logprobs_backward(one, None, z, stats, t)
    u = torch.finfo(dtype).eps / 2
    q = math.exp(-d) / s
    assert float((grad[:, 3].double() - (1 - 1 / s)).abs().max()) <= u * (1 - 1 / s) + 2.0 ** -14 / s + 2.0 ** -23
    assert float((grad[:, 4].double() + q).abs().max()) <= (u + 2.0 ** -13) * q
