"""CPU checks of the tensor helpers of the embedding, the linear recurrence and
the cross entropy of a linear layer: which device is current, and on which
stream they copy, when the library is called (a recorder stands in for the
library; no kernel is launched)."""
import pytest

torch = pytest.importorskip("torch")


class Recorder:
    """The library, as long as the tensors' device is current."""

    def __init__(self):
        self.inside, self.calls, self.outside = 0, [], []

    def __enter__(self):
        self.inside += 1

    def __exit__(self, *_):
        self.inside -= 1

    def __getattr__(self, name):
        def call(*args):
            (self.calls if self.inside else self.outside).append(name)
            return 0
        return call


@pytest.fixture
def seq(fg_lib):
    from fft_convolution_gb300 import sequence
    return sequence


@pytest.fixture
def recorder(seq, monkeypatch):
    """The helpers on tensors without memory, whose device is not current."""
    rec = Recorder()
    monkeypatch.setattr(seq, "_lib", rec)
    monkeypatch.setattr(seq, "_device", lambda *tensors: torch.device("meta"))
    monkeypatch.setattr(seq, "_current", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda device: rec)
    return rec


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, device="meta", dtype=dtype)


def calls(seq):
    """Every helper once, on strided inputs."""
    ids, table, dy = meta(6, 8, dtype=torch.int64)[:, ::2], meta(30, 64)[:, ::2], meta(6, 4, 64)[..., ::2]
    yield "fft_embedding", lambda: seq.embedding(ids, table)
    yield "fft_embedding_backward", lambda: seq.embedding_backward(dy, ids, 30)
    yield "fft_embedding_backward", lambda: seq.embedding_backward(dy, ids, 30, add_to=meta(30, 32))
    x, state = meta(2, 5, 64)[..., ::2], meta(2, 64)[:, ::2]
    offsets = torch.empty(6, dtype=torch.int64, device="meta")[::2]
    yield "fft_linear_recurrence", lambda: seq.linear_recurrence(x, x, x, initial_state=state)
    yield "fft_linear_recurrence", lambda: seq.linear_recurrence(x[0], x[0], initial_state=state, offsets=offsets)
    yield "fft_linear_recurrence_backward", lambda: seq.linear_recurrence_backward(
        x, x, x, x, beta=x, initial_state=state, dfinal_state=state)
    yield "fft_linear_recurrence_step", lambda: seq.linear_recurrence_step(x, x, meta(3, 32), beta=x)
    rows, targets, losses = meta(10, 64)[:, ::2], meta(20, dtype=torch.int64)[::2], meta(20)[::2]
    yield "fft_linear_cross_entropy", lambda: seq.linear_cross_entropy(rows, table, targets)
    yield "fft_linear_cross_entropy_backward", lambda: seq.linear_cross_entropy_backward(losses, rows, table, targets, losses)


def test_the_tensors_device_is_current_in_every_call(seq, recorder):
    for name, call in calls(seq):
        recorder.calls.clear()
        call()
        assert name in recorder.calls and not recorder.outside, name
        assert recorder.inside == 0


def test_copies_belong_to_the_calls_stream(seq, recorder, monkeypatch):
    contiguous, outside = torch.Tensor.contiguous, []

    def watched(t, *args, **kwargs):
        if not recorder.inside:
            outside.append(tuple(t.shape))
        return contiguous(t, *args, **kwargs)
    monkeypatch.setattr(torch.Tensor, "contiguous", watched)
    for name, call in calls(seq):
        call()
        assert not outside, name


def test_public_names(fg_lib):
    for name in ("embedding", "embedding_backward", "linear_recurrence", "linear_recurrence_backward",
                 "linear_recurrence_step", "linear_cross_entropy", "linear_cross_entropy_backward"):
        assert callable(getattr(fg_lib, name))
