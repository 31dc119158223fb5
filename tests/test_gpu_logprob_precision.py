"""What the sums of the log probabilities keep: errors against 64 bits beside those of elementary fp32 operations, signs of
log probabilities and entropies, and rows of very many logits."""
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
