"""Which workspaces the operators of a training step accept from their caller, without a GPU: contiguous tensors on the GPU of
the operands, with as many bytes behind their first multiple of 256 as are needed."""
import pytest

torch = pytest.importorskip("torch")

import orthogonalized_optimizer_step_amd.train_ops as T  # noqa: E402
from orthogonalized_optimizer_step_amd._lib import DionError  # noqa: E402


class Given:
    def __init__(self, device=0, at=4096, count=5000, size=1, contiguous=True):
        self.device, self.at, self.count, self.size, self.contiguous = device, at, count, size, contiguous

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.count

    def element_size(self):
        return self.size


@pytest.mark.parametrize("take", [T._workspace, T._scratch])
@pytest.mark.parametrize("given,fits", [
    (Given(), (4096, 5000)), (Given(at=4097), (4352, 4745)), (Given(count=512), (4096, 512)),
    (Given(count=128, size=4), (4096, 512)), (Given(at=4097, count=767), (4352, 512)),
    (Given(at=4097, count=766), None), (Given(count=511), None), (Given(contiguous=False), None),
    (Given(device=1), None),    # another GPU's memory
    (Given(device=-1), None)])  # the host's
def test_given_workspaces(take, given, fits):
    if fits is None:
        with pytest.raises(DionError):
            take(512, Given(), given, None)
    else:
        assert take(512, Given(), given, None) == (given, *fits)
