"""The linear recurrence with its states in place: final_state is initial_state, and
dinitial_state is dfinal_state, which the C ABI allows.  The same bits as with
arrays of their own, for one block per sequence and for clusters of them (every
block of which reads the state that one of them overwrites)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_recurrence import TYPES, inputs  # noqa: E402

CODES = {"f32": 0, "bf16": 2, "f16": 3}


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("kind,gated", [("f32", True), ("bf16", False), ("f16", True)])
@pytest.mark.parametrize("batch,tokens,channels,offsets", [
    (1, 4000, 64, None), (1, 1025, 7, None), (2, 130, 260, None), (1, 1, 40, None), (3, 0, 40, None),  # clusters
    (200, 300, 128, None), (200, 60, 33, None),                                                        # a block each
    (4, 3000, 96, [0, 0, 1700, 1701, 3000]), (2, 500, 45, [100, 450, 450])])
def test_states_in_place(fg, batch, tokens, channels, offsets, kind, gated):
    shape = (tokens, channels) if offsets else (batch, tokens, channels)
    x, g, beta, _, dy, _ = inputs(batch + tokens, shape, TYPES[kind], TYPES[kind], gated)
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda") if offsets else None
    d = fg.RecurrenceDesc(batch, tokens, channels)
    for n in ("x", "g", "beta"):
        setattr(d, n + "_stride", (tokens * channels, channels))
    d.dtype = d.gtype = CODES[kind]
    d.clear_rows = 1
    stream = torch.cuda.current_stream().cuda_stream
    h0, d1 = torch.randn(batch, channels, device="cuda"), torch.randn(batch, channels, device="cuda")
    y, final = fg.linear_recurrence(x, g, beta, initial_state=h0, offsets=at)
    dx, dg, db, d0 = fg.linear_recurrence_backward(dy, x, g, y, beta=beta, initial_state=h0, offsets=at, dfinal_state=d1)
    for _ in range(20):
        state, grad = h0.clone(), d1.clone()
        y2, dx2, dg2, db2 = (None if t is None else torch.empty_like(t) for t in (y, dx, dg, db))
        assert fg.fft_linear_recurrence(d, x.data_ptr(), g.data_ptr(), ptr(beta), ptr(at), state.data_ptr(), y2.data_ptr(),
                                        state.data_ptr(), None, 0, stream) == 0
        assert torch.equal(y2, y) and torch.equal(state, final)
        assert fg.fft_linear_recurrence_backward(d, dy.data_ptr(), x.data_ptr(), g.data_ptr(), ptr(beta), y2.data_ptr(),
                                                 ptr(at), h0.data_ptr(), grad.data_ptr(), dx2.data_ptr(), dg2.data_ptr(),
                                                 ptr(db2), grad.data_ptr(), None, 0, stream) == 0
        assert torch.equal(grad, d0) and torch.equal(dx2, dx) and torch.equal(dg2, dg)
        assert db is None or torch.equal(db2, db)
