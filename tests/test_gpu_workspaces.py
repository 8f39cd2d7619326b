"""Workspaces on any 16-byte boundary, which is all that the C ABI asks for: the
cross entropy of a linear layer, the embedding's gradient and the recurrence
of many packed sequences give the same bits as on a 256-byte boundary, and write
nothing outside."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_model_guards import CODES, TYPES, Guarded, stream  # noqa: E402


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


SHIFTS = [16, 32, 112, 240]


# G alone; sums of dx cut into slices; sums of dW; several pieces of the words
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("tokens,vocabulary,dim", [(1, 1, 1), (40, 300, 64), (300, 2100, 136), (20000, 70, 24), (60000, 4353, 8)])
def test_cross_entropy(fg, kind, shift, tokens, vocabulary, dim):
    t, code = TYPES[kind], CODES[kind]
    x, w = torch.randn(tokens, dim, device="cuda").to(t), torch.randn(vocabulary, dim, device="cuda").to(t)
    targets = torch.randint(-1, vocabulary, (tokens,), device="cuda")
    dloss = torch.rand(tokens, device="cuda")
    sizes = [fg.fft_linear_cross_entropy_workspace_bytes(x.data_ptr(), dim, w.data_ptr(), dim, tokens, vocabulary, dim, code,
                                                         back) for back in (0, 1)]
    ws, back = (Guarded(n, shift) for n in sizes)
    loss, lse = Guarded(4 * tokens), Guarded(4 * tokens)
    dx, dw = Guarded(tokens * dim * t.itemsize), Guarded(vocabulary * dim * t.itemsize)
    assert fg.fft_linear_cross_entropy(x.data_ptr(), dim, w.data_ptr(), dim, targets.data_ptr(), 8, loss.ptr, lse.ptr, tokens,
                                       vocabulary, dim, code, ws.ptr, ws.nbytes, stream()) == 0
    assert fg.fft_linear_cross_entropy_backward(dloss.data_ptr(), x.data_ptr(), dim, w.data_ptr(), dim, targets.data_ptr(), 8,
                                                lse.ptr, dx.ptr, dw.ptr, tokens, vocabulary, dim, code, back.ptr, back.nbytes,
                                                stream()) == 0
    for b in (loss, lse, dx, dw, ws, back):
        assert b.intact()
    want, sums = fg.linear_cross_entropy(x, w, targets)
    assert torch.equal(loss.values(torch.float32, tokens), want) and torch.equal(lse.values(torch.float32, tokens), sums)
    gx, gw = fg.linear_cross_entropy_backward(dloss, x, w, targets, sums)
    assert torch.equal(dx.values(t, tokens, dim), gx) and torch.equal(dw.values(t, vocabulary, dim), gw)
    assert fg.fft_device_status(None) == fg.FFT_OK


@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("kind", list(TYPES))
def test_embedding_gradient(fg, kind, shift):
    t, code, tokens, rows, dim = TYPES[kind], CODES[kind], 3000, 90, 64
    dy, ids = torch.randn(tokens, dim, device="cuda").to(t), torch.randint(-2, rows + 2, (tokens,), device="cuda")
    grad, ws = Guarded(rows * dim * t.itemsize), Guarded(fg.fft_embedding_workspace_bytes(tokens, dim, code), shift)
    assert fg.fft_embedding_backward(dy.data_ptr(), dim, ids.data_ptr(), 8, grad.ptr, tokens, rows, dim, 2.0, 0, code, code,
                                     ws.ptr, ws.nbytes, stream()) == 0
    assert grad.intact() and ws.intact()
    assert torch.equal(grad.values(t, rows, dim), fg.embedding_backward(dy, ids, rows, scale=2.0))


@pytest.mark.parametrize("shift", SHIFTS)
def test_packed_recurrence(fg, shift):
    sequences, tokens, channels = 1500, 4000, 40
    x, g = torch.randn(tokens, channels, device="cuda"), -torch.rand(tokens, channels, device="cuda")
    cuts = torch.randint(0, tokens + 1, (sequences + 1,), device="cuda").sort()[0].int()
    d = fg.RecurrenceDesc(sequences, tokens, channels)
    for n in ("x", "g", "beta"):
        setattr(d, n + "_stride", (0, channels))
    d.clear_rows = 1
    y, last = Guarded(4 * tokens * channels), Guarded(4 * sequences * channels)
    ws = Guarded(fg.fft_linear_recurrence_workspace_bytes(d, 1), shift)
    assert fg.fft_linear_recurrence(d, x.data_ptr(), g.data_ptr(), None, cuts.data_ptr(), None, y.ptr, last.ptr, ws.ptr,
                                    ws.nbytes, stream()) == 0
    assert y.intact() and last.intact() and ws.intact()
    want, final = fg.linear_recurrence(x, g, offsets=cuts)
    assert torch.equal(y.values(torch.float32, tokens, channels), want)
    assert torch.equal(last.values(torch.float32, sequences, channels), final)
