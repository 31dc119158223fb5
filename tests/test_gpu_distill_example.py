"""The example that runs the training-step operators together with the optimizer: the student learns."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_distillation_example_learns():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("distill_example", os.path.join(ROOT, "examples", "distill.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(steps=25, tokens=512, vocab=1001, k=32)
    assert all(math.isfinite(v) for v in losses)
    # a student that knows nothing is T^2 log(vocab) less the teacher's entropy away; it has to lose a quarter
    assert losses[-1] < 0.75 * losses[0], losses
