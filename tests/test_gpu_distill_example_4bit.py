"""The distillation example with a layer-norm model and a teacher in 4 bits: it runs, and the gradients of its step are
those of the same step in float64 with automatic differentiation."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_4_bit_example_runs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("distill_example", os.path.join(ROOT, "examples", "distill.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(steps=3, tokens=256, vocab=1001, k=16, bits=4)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


def test_the_gradients_of_its_step():
    """fp32 leaves, so that only the operators' own roundings count: sums of up to 600 fp32 terms (2^-14 of the
    magnitudes if all errors point one way) and two fp32 matrix products with 64 and 600 terms.  2^-11 of each gradient's
    largest element allows for both."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import orthogonalized_optimizer_step_amd as dion
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tokens, dim, vocab, k, T = 40, 64, 600, 8, 2.0
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x, layer, norm, shift, head = randn(tokens, dim), randn(dim, dim) / 8, randn(dim), randn(dim), randn(vocab, dim) * 0.1
    codes, scale = dion.mxfp4_quantize(dion.layernorm(x @ layer, norm, shift, residual=x)[0])
    hq, hs = dion.mxfp4_quantize(randn(vocab, dim))
    top, index = dion.top_logprobs(dion.mxfp4_linear(codes, scale, hq, hs, out_dtype=torch.float32), k)[:2]
    index[:5] = -1
    leaves = [t.clone().requires_grad_() for t in (layer, norm, shift, head)]
    y, _ = dion.layer_norm(x @ leaves[0].t(), leaves[1], leaves[2], x)
    logits = y @ leaves[3].t()
    logprob, entropy = dion.log_probs(logits, index[:, 0])
    (dion.distill_loss(logits, top, index, T) - 0.1 * logprob - 0.001 * entropy * (index[:, 0] >= 0)).sum().backward()
    # the same in float64, from torch's elementary operations
    X = x.double()
    L, N, S, H = (t.double().clone().requires_grad_() for t in (layer, norm, shift, head))
    s = X @ L.t() + X
    d = s - s.mean(1, keepdim=True)
    Y = d / (d.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * N + S
    Z = Y @ H.t()
    live = index[:, 0] >= 0
    p = torch.softmax(top.double() / T, 1)
    logq = torch.log_softmax(Z / T, 1).gather(1, index.clamp_min(0))
    loss = T * T * (p * (p.log() - logq)).sum(1) * live
    logq1 = torch.log_softmax(Z, 1)
    lp = logq1.gather(1, index[:, :1].clamp_min(0))[:, 0] * live
    ent = -(logq1.exp() * logq1).sum(1)
    (loss - 0.1 * lp - 0.001 * ent * live).sum().backward()
    for a, b in zip(leaves, (L, N, S, H)):
        assert (a.grad.double() - b.grad).abs().max() <= 2.0 ** -11 * b.grad.abs().max()
