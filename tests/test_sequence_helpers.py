"""CPU checks of the tensor helpers of the sequence-model operators: which
device is current, and on which stream they copy, when the library is
called (a recorder stands in for the library; no kernel is launched)."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def seq(fg_lib):
    from fft_convolution_gb300 import sequence
    return sequence


def test_device_and_stream_of_a_call(seq, monkeypatch):
    zero, one = torch.device("cuda", 0), torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(seq, "_current", lambda index: 100 + index)
    context, handle = seq._on(None, one)
    assert isinstance(context, torch.cuda.device) and context.idx == 1 and handle == 101
    context, handle = seq._on(None, zero)
    assert context is seq._NULL and handle == 100
    with pytest.raises(ValueError):
        seq._on(types.SimpleNamespace(device=zero, cuda_stream=7), one)


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
def recorder(seq, monkeypatch):
    """The helpers on tensors without memory, whose device is not current."""
    rec = Recorder()
    monkeypatch.setattr(seq, "_lib", rec)
    monkeypatch.setattr(seq, "_device", lambda *tensors: torch.device("meta"))
    monkeypatch.setattr(seq, "_table", lambda tensors, what: (*(seq.array.array("q", [1]),) * 3, torch.device("meta")))
    monkeypatch.setattr(seq, "_current", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda device: rec)
    return rec


def meta(*shape):
    return torch.empty(*shape, device="meta")


def calls(seq):
    """Every helper once, on strided inputs."""
    x, w, stats = meta(5, 32)[:, ::2], meta(32)[::2], meta(10)[::2]
    yield "fft_layer_norm", lambda: seq.layer_norm(x, w, w)
    yield "fft_layer_norm_backward", lambda: seq.layer_norm_backward(x, x, w, stats, stats)
    yield "fft_grad_norm", lambda: seq.grad_norm([x])
    yield "fft_clip_grad_norm", lambda: seq.clip_grad_norm([x], 1.0)
    q, v, g = meta(2, 3, 1, 32)[..., ::2], meta(2, 3, 2, 16)[..., ::2], meta(2, 3, 2)
    state, slots = meta(2, 2, 16, 16)[..., ::2], torch.empty(2, dtype=torch.int32, device="meta")
    offsets = torch.empty(6, dtype=torch.int64, device="meta")[::2]
    yield "fft_delta_rule", lambda: seq.delta_rule(q, q, v, g, g, initial_state=state)
    yield "fft_delta_rule", lambda: seq.delta_rule(q[0], q[0], v[0], g[0], g[0], initial_state=state, offsets=offsets)
    yield "fft_delta_rule_backward", lambda: seq.delta_rule_backward(v, q, q, v, g, g, initial_state=state,
                                                                     dfinal_state=state)
    yield "fft_delta_rule_step", lambda: seq.delta_rule_step(q, q, v, g, g, meta(2, 2, 16, 8), slots=slots)


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
