"""CPU checks of the C ABI of the embedding, the gated linear recurrence and
the cross entropy of a linear layer: arguments that make no sense are refused
before anything is enqueued (no kernel is launched by any call here), sizes of
nothing are accepted, workspaces are sized on the host."""
import pytest

P = 4096  # an address that is never looked at


@pytest.fixture(scope="module")
def fg(fg_lib):
    return fg_lib


def lookup(fg, ids=P, id_bytes=8, table=P, ldt=8, y=P, ldy=8, tokens=2, rows=5, dim=8, scale=1.0, dtype=0):
    return fg.fft_embedding(ids, id_bytes, table, ldt, y, ldy, tokens, rows, dim, scale, dtype, None)


SIZES = [(dict(tokens=-1), 1), (dict(rows=0), 1), (dict(dim=0), 1), (dict(dtype=4), 1), (dict(dtype=-1), 1),
         (dict(id_bytes=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
         (dict(tokens=2 ** 31 - 63), 3), (dict(rows=2 ** 31), 3), (dict(rows=2 ** 30, dim=2 ** 20), 3)]


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(ids=None), 1), (dict(table=None), 1), (dict(y=None), 1), (dict(ldt=7), 1), (dict(ldy=7), 1),
    (dict(ldt=2 ** 62), 3), (dict(ids=P + 4), 6), (dict(ids=P + 2, id_bytes=4), 6), (dict(table=P + 2), 6),
    (dict(y=P + 2), 6), (dict(dtype=1, y=P + 4), 6)])
def test_embedding_refuses(fg, change, status):
    assert lookup(fg, **change) == status


def grad(fg, dy=P, lddy=8, ids=P, id_bytes=8, dtable=P, tokens=2, rows=5, dim=8, scale=1.0, add=0, dtype=0, ttype=None,
         ws=P, nbytes=1 << 40):
    return fg.fft_embedding_backward(dy, lddy, ids, id_bytes, dtable, tokens, rows, dim, scale, add, dtype,
                                     dtype if ttype is None else ttype, ws, nbytes, None)


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(dy=None), 1), (dict(ids=None), 1), (dict(dtable=None), 1), (dict(ws=None), 1), (dict(lddy=7), 1), (dict(ttype=9), 1),
    (dict(nbytes=100), 1), (dict(dtype=0, ttype=2), 3), (dict(dtype=2, ttype=3), 3), (dict(dtype=1, ttype=0), 3),
    (dict(lddy=2 ** 62), 3), (dict(tokens=2 ** 30, dim=2 ** 15, lddy=2 ** 15), 3), (dict(dtable=P + 2), 6), (dict(ws=P + 8), 6), (dict(dy=P + 2), 6), (dict(ids=P + 4), 6)])
def test_embedding_backward_refuses(fg, change, status):
    assert grad(fg, **change) == status


def test_embedding_of_nothing(fg):
    assert lookup(fg, tokens=0, ids=None, table=None, y=None) == fg.FFT_OK
    assert grad(fg, tokens=0, dy=None, ids=None, ws=None, nbytes=0, add=1) == fg.FFT_OK
    assert fg.fft_embedding_workspace_bytes(0, 8, 0) == 0
    assert fg.fft_embedding_workspace_bytes(-1, 8, 0) == 0
    need = fg.fft_embedding_workspace_bytes(1000, 8, 0)
    assert need >= 16 * 1000 and grad(fg, tokens=1000, nbytes=need - 1) == fg.FFT_ERR_INVALID_ARG


def desc(fg, **change):
    a = dict(batch=2, tokens=10, channels=24, dtype=0, gtype=0, clear_rows=0)
    a.update(change)
    d = fg.RecurrenceDesc(*(a[n] for n in ("batch", "tokens", "channels")))
    for n in ("x", "g", "beta"):
        setattr(d, n + "_stride", a.get(n + "_stride", (1000, 100)))
    d.dtype, d.gtype, d.clear_rows = a["dtype"], a["gtype"], a["clear_rows"]
    return d


def forward(fg, d, x=P, g=P, beta=P, offsets=None, s0=None, y=P, s1=P, ws=None, nbytes=0):
    return fg.fft_linear_recurrence(d, x, g, beta, offsets, s0, y, s1, ws, nbytes, None)


def backward(fg, d, dy=P, x=P, g=P, beta=P, y=P, offsets=None, s0=None, d1=None, dx=P, dg=P, db=P, d0=P, ws=None,
             nbytes=0):
    return fg.fft_linear_recurrence_backward(d, dy, x, g, beta, y, offsets, s0, d1, dx, dg, db, d0, ws, nbytes, None)


def step(fg, d, x=P, g=P, beta=P, state=P, slots=None, pool=2, y=P):
    return fg.fft_linear_recurrence_step(d, x, g, beta, state, slots, pool, y, None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), 1), (dict(tokens=-1), 1), (dict(channels=0), 1), (dict(dtype=7), 1), (dict(gtype=-1), 1),
    (dict(x_stride=(1, -1)), 1), (dict(g_stride=(-1, 1)), 1), (dict(dtype=1, gtype=1), 3), (dict(dtype=0, gtype=2), 3),
    (dict(dtype=2, gtype=3), 3), (dict(batch=2 ** 24 + 1), 3), (dict(tokens=2 ** 31), 3), (dict(channels=2 ** 30 + 1), 3),
    (dict(batch=2 ** 24, channels=2 ** 20), 3), (dict(batch=2 ** 16, tokens=2 ** 25, channels=2 ** 6), 3)])
def test_recurrence_refuses_sizes(fg, change, status):
    d = desc(fg, **change)
    assert forward(fg, d) == status and backward(fg, d) == status and step(fg, d, pool=1 << 40) == status


@pytest.mark.parametrize("name", ["x", "g", "y"])
def test_recurrence_refuses_missing(fg, name):
    assert forward(fg, desc(fg), **{name: None}) == fg.FFT_ERR_INVALID_ARG
    assert step(fg, desc(fg), **{name: None}) == fg.FFT_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["x", "g", "beta", "y", "s0", "s1", "offsets"])
def test_recurrence_refuses_misaligned(fg, name):
    assert forward(fg, desc(fg), **{name: P + 2}) == fg.FFT_ERR_MISALIGNED


@pytest.mark.parametrize("name", ["dy", "x", "g", "y", "dx", "dg", "db"])
def test_recurrence_backward_refuses(fg, name):
    assert backward(fg, desc(fg), **{name: None}) == fg.FFT_ERR_INVALID_ARG
    assert backward(fg, desc(fg), **{name: P + 2}) == fg.FFT_ERR_MISALIGNED


@pytest.mark.parametrize("name", ["offsets", "s0", "d1", "d0"])
def test_recurrence_backward_refuses_misaligned(fg, name):
    assert backward(fg, desc(fg), **{name: P + 2}) == fg.FFT_ERR_MISALIGNED


def test_recurrence_step_refuses(fg):
    d = desc(fg)
    assert step(fg, d, pool=1) == fg.FFT_ERR_INVALID_ARG       # two sequences, one state
    assert step(fg, d, pool=-1, slots=P) == fg.FFT_ERR_INVALID_ARG
    assert step(fg, d, state=None) == fg.FFT_ERR_INVALID_ARG
    assert step(fg, d, slots=P + 2) == fg.FFT_ERR_MISALIGNED
    assert step(fg, d, state=P + 2) == fg.FFT_ERR_MISALIGNED
    assert fg._lib.fft_linear_recurrence(None, P, P, P, None, None, P, P, None, 0, None) == fg.FFT_ERR_INVALID_ARG


def test_recurrence_workspaces(fg):
    few, many = desc(fg, batch=1024), desc(fg, batch=1025)
    size = fg.fft_linear_recurrence_workspace_bytes
    assert size(few, 1) == 0 and size(many, 0) == 0 and size(desc(fg, channels=0), 1) == 0
    need = size(many, 1)
    assert need >= 1026 * 4
    for call in (forward, backward):
        assert call(fg, many, offsets=P, ws=P, nbytes=need - 1) == fg.FFT_ERR_INVALID_ARG
        assert call(fg, many, offsets=P, nbytes=need) == fg.FFT_ERR_INVALID_ARG
        assert call(fg, many, offsets=P, ws=P + 8, nbytes=need) == fg.FFT_ERR_MISALIGNED


def test_recurrence_of_nothing(fg):
    none = dict(x=None, g=None, y=None)
    assert forward(fg, desc(fg, batch=0), **none) == fg.FFT_OK
    assert backward(fg, desc(fg, batch=0), dy=None, dx=None, dg=None, **none) == fg.FFT_OK
    assert step(fg, desc(fg, batch=0), **none) == fg.FFT_OK
    assert step(fg, desc(fg, tokens=0), **none) == fg.FFT_OK


def loss(fg, x=P, ldx=8, w=P, ldw=8, targets=P, tbytes=8, loss=P, lse=P, tokens=3, vocabulary=5, dim=8, dtype=0, ws=P,
         nbytes=1 << 50):
    return fg.fft_linear_cross_entropy(x, ldx, w, ldw, targets, tbytes, loss, lse, tokens, vocabulary, dim, dtype, ws, nbytes,
                                       None)


def loss_grad(fg, dloss=P, x=P, ldx=8, w=P, ldw=8, targets=P, tbytes=8, lse=P, dx=P, dw=P, tokens=3, vocabulary=5, dim=8,
              dtype=0, ws=P, nbytes=1 << 50):
    return fg.fft_linear_cross_entropy_backward(dloss, x, ldx, w, ldw, targets, tbytes, lse, dx, dw, tokens, vocabulary, dim,
                                                dtype, ws, nbytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(vocabulary=0), 1), (dict(dim=0), 1), (dict(dtype=4), 1), (dict(tbytes=3), 1), (dict(ldx=7), 1),
    (dict(ldw=7), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(targets=None), 1), (dict(lse=None), 1), (dict(ws=None), 1),
    (dict(nbytes=10), 1), (dict(dtype=1), 3), (dict(tokens=2 ** 24 + 1), 3), (dict(vocabulary=2 ** 24 + 1), 3),
    (dict(dim=2 ** 20 + 1, ldx=2 ** 21, ldw=2 ** 21), 3), (dict(ldx=2 ** 32), 3), (dict(tokens=2 ** 24, vocabulary=2 ** 24), 3),
    (dict(x=P + 2), 6), (dict(w=P + 2), 6), (dict(targets=P + 4), 6), (dict(lse=P + 2), 6), (dict(ws=P + 8), 6)])
def test_cross_entropy_refuses(fg, change, status):
    assert loss(fg, **change) == status
    assert loss_grad(fg, **change) == status


def test_cross_entropy_refuses_more(fg):
    assert loss(fg, loss=None) == fg.FFT_ERR_INVALID_ARG and loss(fg, loss=P + 1) == fg.FFT_ERR_MISALIGNED
    assert loss_grad(fg, dloss=None) == fg.FFT_ERR_INVALID_ARG and loss_grad(fg, dloss=P + 2) == fg.FFT_ERR_MISALIGNED
    assert loss_grad(fg, dx=P + 2) == fg.FFT_ERR_MISALIGNED and loss_grad(fg, dw=P + 2) == fg.FFT_ERR_MISALIGNED


def test_cross_entropy_of_nothing(fg):
    assert loss(fg, tokens=0, x=None, w=None, loss=None, ws=None, nbytes=0) == fg.FFT_OK
    assert loss_grad(fg, dx=None, dw=None, x=None, ws=None, nbytes=0) == fg.FFT_OK
    assert loss_grad(fg, tokens=0, dw=None, x=None, ws=None, nbytes=0) == fg.FFT_OK


def test_cross_entropy_workspaces(fg):
    size = lambda x=P, ldx=64, dtype=2, back=0, n=1000, v=7000: (  # noqa: E731
        fg.fft_linear_cross_entropy_workspace_bytes(x, ldx, P, 64, n, v, 64, dtype, back))
    plain = size()
    assert plain >= 1000 * 55 * 8
    assert size(x=P + 2) >= plain + 1000 * 128     # a copy of rows off their boundaries
    assert size(ldx=65) >= plain + 1000 * 128
    assert size(dtype=0) >= plain + 8000 * 384     # three parts
    assert size(back=1) >= 1000 * 7000 * 2
    # G is bounded: not the logits of 4 * 10^9 values
    assert size(back=1, n=65536, v=65536) <= (256 << 20) + 65536 * 64 * 6 + 65536 * 1024
    assert size(n=-1) == 0 and size(dtype=1) == 0 and size(n=0) == 0
