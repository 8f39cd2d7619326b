"""Nothing outside an output or a workspace is written: the embedding, the linear
recurrence and the cross entropy of a linear layer through the C ABI, every
output and the workspace (of exactly the bytes asked for) inside a larger
allocation whose margins hold a pattern."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

MARGIN = 4096
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": 0, "bf16": 2, "f16": 3}


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


class Guarded:
    """Bytes between two margins; `shift` moves them off their 256-byte boundary."""

    def __init__(self, nbytes, shift=0):
        self.begin, self.nbytes = MARGIN + shift, int(nbytes)
        self.memory = torch.full((self.begin + self.nbytes + MARGIN,), 0xA5, dtype=torch.uint8, device="cuda")

    @property
    def ptr(self):
        return self.memory.data_ptr() + self.begin

    def intact(self):
        return bool((self.memory[:self.begin] == 0xA5).all() and (self.memory[self.begin + self.nbytes:] == 0xA5).all())

    def values(self, dtype, *shape):
        return self.memory[self.begin:self.begin + self.nbytes].clone().view(dtype).reshape(shape)


def stream():
    return torch.cuda.current_stream().cuda_stream


SHIFTS = [0, 16, 4]  # whole vectors, vectors off 32 bytes, elements only


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("tokens,rows,dim", [(1, 1, 1), (50, 7, 33), (300, 90, 64), (1000, 2000, 40), (70000, 30, 8)])
def test_embedding(fg, kind, shift, tokens, rows, dim):
    t, code = TYPES[kind], CODES[kind]
    table, dy = torch.randn(rows, dim, device="cuda").to(t), torch.randn(tokens, dim, device="cuda").to(t)
    ids = torch.randint(-2, rows + 2, (tokens,), device="cuda")
    y, grad = Guarded(tokens * dim * t.itemsize, shift), Guarded(rows * dim * t.itemsize, shift)
    ws = Guarded(fg.fft_embedding_workspace_bytes(tokens, dim, code))
    assert fg.fft_embedding(ids.data_ptr(), 8, table.data_ptr(), dim, y.ptr, dim, tokens, rows, dim, 2.0, code, stream()) == 0
    assert fg.fft_embedding_backward(dy.data_ptr(), dim, ids.data_ptr(), 8, grad.ptr, tokens, rows, dim, 2.0, 0, code, code,
                                     ws.ptr, ws.nbytes, stream()) == 0
    assert y.intact() and grad.intact() and ws.intact()
    assert torch.equal(y.values(t, tokens, dim), fg.embedding(ids, table, scale=2.0))
    want = fg.embedding_backward(dy, ids, rows, scale=2.0)
    assert torch.equal(grad.values(t, rows, dim), want)
    assert fg.fft_embedding_backward(dy.data_ptr(), dim, ids.data_ptr(), 8, grad.ptr, tokens, rows, dim, 2.0, 1, code, code,
                                     ws.ptr, ws.nbytes, stream()) == 0
    assert grad.intact() and ws.intact()
    # the sum and the gradient that it is added to are each rounded once, half a step of at most |twice|; 1e-6 covers the
    # steps below the smallest normal number of a half, 2^-24
    twice = (2 * want.double()).to(t).double()
    assert ((grad.values(t, rows, dim).double() - twice).abs() <= torch.finfo(t).eps * twice.abs() + 1e-6).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("tokens,channels", [(1, 1), (37, 40), (200, 132), (1500, 24), (700, 45)])
def test_recurrence(fg, kind, shift, tokens, channels):
    t, code = TYPES[kind], CODES[kind]
    x, dy = (torch.randn(2, tokens, channels, device="cuda").to(t) for _ in range(2))
    g, beta = -torch.rand(2, tokens, channels, device="cuda").to(t), torch.rand(2, tokens, channels, device="cuda").to(t)
    d = fg.RecurrenceDesc(2, tokens, channels)
    for n in ("x", "g", "beta"):
        setattr(d, n + "_stride", (tokens * channels, channels))
    d.dtype = d.gtype = code
    size, state = 2 * tokens * channels * t.itemsize, 2 * channels * 4
    y, dx, dg, db = (Guarded(size, shift) for _ in range(4))
    last, first, pool = Guarded(state, 4), Guarded(state, 4), Guarded(state, 4)
    assert fg.fft_linear_recurrence(d, x.data_ptr(), g.data_ptr(), beta.data_ptr(), None, None, y.ptr, last.ptr, None, 0,
                                    stream()) == 0
    assert fg.fft_linear_recurrence_backward(d, dy.data_ptr(), x.data_ptr(), g.data_ptr(), beta.data_ptr(), y.ptr, None, None,
                                             None, dx.ptr, dg.ptr, db.ptr, first.ptr, None, 0, stream()) == 0
    for b in (y, dx, dg, db, last, first):
        assert b.intact()
    want, final = fg.linear_recurrence(x, g, beta)
    # two roundings of half a step each, of sums that may be taken in another order: a decay is off by 2^-22 of it, and with
    # decays of 0.63 on average sum_k k a^k |x| is below 8 * 6, so the sums differ by about 48 * 2^-22, 1.2e-5
    eps = torch.finfo(t).eps
    close = lambda a, b: ((a.double() - b.double()).abs() <= eps * b.double().abs() + 1e-4).all()  # noqa: E731
    assert close(y.values(t, 2, tokens, channels), want) and close(last.values(torch.float32, 2, channels), final)
    pool.memory[pool.begin:pool.begin + pool.nbytes] = 0
    one = Guarded(size, shift)
    assert fg.fft_linear_recurrence_step(d, x.data_ptr(), g.data_ptr(), beta.data_ptr(), pool.ptr, None, 2, one.ptr,
                                         stream()) == 0
    assert one.intact() and pool.intact() and close(one.values(t, 2, tokens, channels), want)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shift", SHIFTS)
@pytest.mark.parametrize("tokens,vocabulary,dim", [(1, 1, 1), (40, 300, 33), (129, 257, 64), (500, 1000, 40), (300, 2100, 136),
                                                   (20000, 70, 24)])
def test_cross_entropy(fg, kind, shift, tokens, vocabulary, dim):
    t, code = TYPES[kind], CODES[kind]
    x, w = torch.randn(tokens, dim, device="cuda").to(t), torch.randn(vocabulary, dim, device="cuda").to(t)
    targets = torch.randint(-1, vocabulary, (tokens,), device="cuda")
    dloss = torch.rand(tokens, device="cuda")
    size = lambda back: fg.fft_linear_cross_entropy_workspace_bytes(x.data_ptr(), dim, w.data_ptr(), dim, tokens, vocabulary,  # noqa: E731
                                                                    dim, code, back)
    loss, lse = Guarded(4 * tokens, 4), Guarded(4 * tokens, 4)
    dx, dw = Guarded(tokens * dim * t.itemsize, shift), Guarded(vocabulary * dim * t.itemsize, shift)
    ws, back = Guarded(size(0)), Guarded(size(1))
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
