"""The 4-bit product of up to 17 tokens at the sizes where it goes from one kernel to another, and where k is split."""
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


def matrix(seed, rows, k, off):
    """Any codes, one scale for all (2^0), and their values; with `off` rows a byte further apart, off 16-byte multiples."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = torch.randint(0, 256, (rows, k // 2 + off), generator=g, device="cuda").to(torch.uint8)[:, :k // 2]
    s = torch.full((rows, (k + 31) // 32), 127, dtype=torch.uint8, device="cuda")
    return q, s, O.mx_values(q.cpu().numpy(), s.cpu().numpy(), k)


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("m", [1, 8, 9, 16, 17])
@pytest.mark.parametrize("n,k", [(8192, 512), (8193, 512), (12288, 512), (12289, 1024), (16385, 512), (512, 8192), (500, 8194),
                                 (70, 8448), (1024, 14336), (2049, 14336), (16, 28672), (4097, 16384)])
def test_products_where_plans_change(dion, m, n, k, off):
    """Values are multiples of a half up to 6: terms are multiples of a quarter up to 36, and 28672 of them are below 2^22
    quarters, so that every sum is exact in fp32 in any order."""
    a, sa, A = matrix(m + k, m, k, off)
    b, sb, B = matrix(n + k, n, k, off)
    y = dion.mxfp4_linear(a, sa, b, sb, out_dtype=torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), A @ B.T)
    assert torch.equal(y, dion.mxfp4_linear(a, sa, b, sb, out_dtype=torch.float32))
