"""The 4-bit product with scales at the ends of their range, 2^-127 and 2^126 or 2^127 against one another, and with results
at the ends of fp32's.  Values are multiples of a half up to 6, so every sum here is exact, and what is compared is equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import model_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dion():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as d
    return d


# every kernel, with operands that lie as it needs them and with rows that are copied first
SIZES = [(1, 70, 1024), (16, 300, 96), (3, 512, 14336), (9, 14336, 512), (24, 70, 1024), (40, 130, 160), (130, 200, 512),
         (700, 900, 1024), (1300, 1100, 544), (2049, 1793, 1024)]


def codes(rng, rows, k, positive=False):
    q = rng.integers(0, 256, (rows, k // 2)).astype(np.uint8)
    return q & 0x77 if positive else q


def product(dion, qa, sa, qb, sb, dtype=torch.float32):
    return dion.mxfp4_linear(*(torch.from_numpy(v).cuda() for v in (qa, sa, qb, sb)), out_dtype=dtype)


def values(q, s, k):
    with np.errstate(all="ignore"):
        return O.mx_values(q, s, k)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_scales_at_their_ends_against_one_another(dion, m, n, k):
    """In turn from block to block, the largest of one operand meet the smallest of the other: their scales' product is
    2^-1 to 2, each term a multiple of 2^-3 up to 72, and a sum of 1024 of them below 2^20 such multiples.  Longer ones
    have scales whose product is 1: terms are multiples of 2^-2 up to 36, 14336 of them below 2^21 such multiples."""
    rng = np.random.default_rng(m + n + k)
    blocks = k // 32
    high, low = np.array([253, 254], np.uint8), np.array([0, 1], np.uint8)
    if k > 1024:
        high, low = high[1:], low[:1]
    turn = np.arange(blocks) % 2 == 0
    sa = np.where(turn, rng.choice(high, (m, blocks)), rng.choice(low, (m, blocks)))
    sb = np.where(turn, rng.choice(low, (n, blocks)), rng.choice(high, (n, blocks)))
    qa, qb = codes(rng, m, k), codes(rng, n, k)
    want = values(qa, sa, k) @ values(qb, sb, k).T
    assert np.array_equal(product(dion, qa, sa, qb, sb).double().cpu().numpy(), want)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("sa,sb", [(0, 127), (127, 0), (0, 128), (1, 110), (60, 67), (254, 103), (110, 240)])
def test_results_at_the_ends_of_fp32(dion, m, n, k, sa, sb):
    """Subnormal results are kept (multiples of 2^-2 2^(sa + sb - 254), 2^-145 or more), and so are large ones (14336 * 36
    2^103, below 2^123, at most)."""
    rng = np.random.default_rng(m + k)
    qa, qb = codes(rng, m, k), codes(rng, n, k)
    one = lambda rows, v: np.full((rows, (k + 31) // 32), v, np.uint8)
    want = values(qa, one(m, 127), k) @ values(qb, one(n, 127), k).T * 2.0 ** (sa + sb - 254)
    got = product(dion, qa, one(m, sa), qb, one(n, sb)).double().cpu().numpy()
    assert np.array_equal(got, want) and np.abs(want).max() < 2.0 ** 127


@pytest.mark.parametrize("m,n,k", SIZES)
def test_results_beyond_fp32(dion, m, n, k):
    """Positive products above its range are infinite, those below it 0."""
    rng = np.random.default_rng(m + k)
    qa, qb = codes(rng, m, k, True) | 0x11, codes(rng, n, k, True) | 0x11   # none is 0
    one = lambda rows, v: np.full((rows, (k + 31) // 32), v, np.uint8)
    assert torch.isposinf(product(dion, qa, one(m, 254), qb, one(n, 254))).all()
    assert not product(dion, qa, one(m, 0), qb, one(n, 0)).any()
