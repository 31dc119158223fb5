"""The Python binding of the training-step operators without a GPU: what it does around its calls."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import orthogonalized_optimizer_step_amd.train_ops as T  # noqa: E402


class Sliced:
    """A tensor that is not contiguous, and says on which stream it is copied and which streams use it."""

    def __init__(self, dtype, streams, log):
        self.shape, self.dtype, self.streams, self.log = (4, 3), dtype, streams, log

    def is_contiguous(self):
        return False

    def contiguous(self):
        self.log.append(("copied", self.streams[-1]))
        return self

    def record_stream(self, stream):
        self.log.append(("used", stream))

    def element_size(self):
        return 8


@pytest.mark.parametrize("stream", [None, "side"])
def test_teacher_copies_are_made_on_the_stream_that_reads_them(monkeypatch, stream):
    streams, log = ["current"], []

    @contextlib.contextmanager
    def on(s):
        streams.append(s)
        yield
        streams.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(T, "_device", lambda *a: 0)
    monkeypatch.setattr(T, "_beside", lambda *a: None)
    monkeypatch.setattr(T, "_matrix", lambda *a: (4, 9, 9))
    T._distill_inputs(torch.zeros(4, 9), Sliced(torch.float32, streams, log), Sliced(torch.int64, streams, log), stream)
    where = stream or "current"
    assert [s for what, s in log if what == "copied"] == [where, where]
    assert [s for what, s in log if what == "used"] == ([] if stream is None else [stream, stream])


@pytest.mark.parametrize("shape,rows", [((2, 3, 0), 6), ((5, 0), 5), ((0, 4, 7), 0), ((2, 0, 7), 0), ((0,), 1), ((4, 1, 0, 0), 0),
                                        ((2, 3, 4), 6), ((7,), 1)])
def test_rows_of_tensors_with_and_without_elements(shape, rows):
    got, cols, ld = T._matrix(torch.zeros(shape), "x")
    assert (got, cols) == (rows, shape[-1]) and ld >= cols
