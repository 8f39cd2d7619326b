"""CPU checks of the sequence-model operators' C ABI: arguments that make no
sense are refused before anything is enqueued (no kernel is launched by any
call here), sizes of nothing are accepted, workspaces are sized on the host."""
import ctypes

import pytest

P = 4096  # an address that is never looked at


@pytest.fixture(scope="module")
def fg(fg_lib):
    return fg_lib


def arrays(n, ptr=P, numel=4, dtype=0):
    return ((ctypes.c_void_p * n)(*[ptr] * n), (ctypes.c_int64 * n)(*[numel] * n), (ctypes.c_int * n)(*[dtype] * n))


def norm(fg, x=P, ldx=8, w=P, b=P, y=2 * P, ldy=8, mean=P, rstd=P, rows=2, dim=8, eps=1e-5, dtype=0, wtype=0):
    return fg.fft_layer_norm(x, ldx, w, b, y, ldy, mean, rstd, rows, dim, eps, dtype, wtype, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(ldx=7), 1), (dict(ldy=7), 1), (dict(rows=-1), 1), (dict(dim=0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dtype=4), 1), (dict(dtype=-1), 1), (dict(wtype=9), 1),
    (dict(x=P, y=P, ldx=8, ldy=9), 1),
    (dict(dtype=0, wtype=2), 3), (dict(dtype=2, wtype=3), 3), (dict(dtype=1, wtype=0), 3),
    (dict(dim=(1 << 30) + 1, ldx=1 << 31, ldy=1 << 31), 3),
    (dict(x=P + 2), 6), (dict(y=P + 1), 6), (dict(w=P + 2), 6), (dict(mean=P + 2), 6),
    (dict(dtype=2, wtype=2, x=P + 1), 6)])
def test_layer_norm_refuses(fg, bad, status):
    assert norm(fg, **bad) == status


def test_layer_norm_of_nothing(fg):
    assert norm(fg, rows=0, x=None, y=None) == fg.FFT_OK


def grad(fg, dy=P, lddy=8, x=P, ldx=8, w=P, mean=P, rstd=P, dx=2 * P, lddx=8, dw=P, db=P, rows=2, dim=8, dtype=0,
         wtype=0, ws=P, nbytes=1 << 30):
    return fg.fft_layer_norm_backward(dy, lddy, x, ldx, w, mean, rstd, dx, lddx, dw, db, rows, dim, dtype, wtype, ws,
                                      nbytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dy=None), 1), (dict(x=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1), (dict(lddy=7), 1),
    (dict(lddx=7), 1), (dict(ws=None), 1), (dict(dx=P, lddx=9), 1), (dict(dim=0), 1), (dict(dtype=5), 1),
    (dict(dtype=3, wtype=2), 3), (dict(dy=P + 2), 6), (dict(dw=P + 1), 6), (dict(ws=P + 8), 6)])
def test_layer_norm_backward_refuses(fg, bad, status):
    assert grad(fg, **bad) == status


def test_layer_norm_backward_of_nothing(fg):
    assert grad(fg, dx=None, dw=None, db=None, ws=None, nbytes=0) == fg.FFT_OK
    assert grad(fg, rows=0, dy=None, x=None, dw=None, db=None, ws=None) == fg.FFT_OK
    assert fg.fft_layer_norm_workspace_bytes(-1, 8, 0) == 0
    assert fg.fft_layer_norm_workspace_bytes(8, 8, 7) == 0


@pytest.mark.parametrize("change,status", [
    (dict(count=-1), 1), (dict(ins=None), 1), (dict(numels=None), 1), (dict(norm=None), 1), (dict(ws=None), 1),
    (dict(dtype=4), 1), (dict(numel=-1), 1), (dict(ptr=None), 1), (dict(ptr=P + 2), 6), (dict(ptr=P + 4, dtype=1), 6),
    (dict(norm=P + 2), 6), (dict(ws=P + 8), 6)])
def test_grad_norm_refuses(fg, change, status):
    a = dict(count=2, norm=P, ws=P, ptr=P, numel=4, dtype=0)
    a.update(change)
    ins, numels, dtypes = arrays(2, a["ptr"], a["numel"], a["dtype"])
    got = fg.fft_grad_norm(a["count"], a.get("ins", ins), a.get("numels", numels), dtypes, a["norm"], a["ws"], 1 << 30,
                           None)
    assert got == status


@pytest.mark.parametrize("change,status", [(dict(max_norm=-1.0), 1), (dict(max_norm=float("nan")), 1),
                                           (dict(eps=-1.0), 1), (dict(outs=None), 1), (dict(out=None), 1),
                                           (dict(out=P + 2), 6)])
def test_clip_refuses(fg, change, status):
    a = dict(max_norm=1.0, eps=1e-6, out=P)
    a.update(change)
    ins, numels, dtypes = arrays(2)
    outs = arrays(2, a["out"])[0] if "outs" not in a else None
    assert fg.fft_clip_grad_norm(2, ins, outs, numels, dtypes, a["max_norm"], a["eps"], P, P, 1 << 30, None) == status


def desc(fg, **change):
    a = dict(batch=2, tokens=10, kheads=2, vheads=4, dk=16, dv=24, scale=0.25, dtype=0)
    a.update(change)
    d = fg.DeltaDesc(*(a[n] for n in ("batch", "tokens", "kheads", "vheads", "dk", "dv")))
    for n in ("q", "k", "v", "g", "beta"):
        setattr(d, n + "_stride", a.get(n + "_stride", (1000, 100, 50)))
    d.scale, d.dtype = a["scale"], a["dtype"]
    return d


def forward(fg, d, q=P, k=P, v=P, g=P, beta=P, offsets=None, s0=None, o=P, s1=P, ws=P, nbytes=1 << 40):
    return fg.fft_delta_rule(d, q, k, v, g, beta, offsets, s0, o, s1, ws, nbytes, None)


def backward(fg, d, do=P, q=P, k=P, v=P, g=P, beta=P, offsets=None, s0=None, ds1=None, dq=P, dk=P, dv=P, dg=P, db=P,
             ds0=P, ws=P, nbytes=1 << 40):
    return fg.fft_delta_rule_backward(d, do, q, k, v, g, beta, offsets, s0, ds1, dq, dk, dv, dg, db, ds0, ws, nbytes,
                                      None)


def step(fg, d, q=P, k=P, v=P, g=P, beta=P, state=P, slots=None, pool=2, o=P):
    return fg.fft_delta_rule_step(d, q, k, v, g, beta, state, slots, pool, o, None)


BAD_SIZES = [(dict(batch=-1), 1), (dict(tokens=-1), 1), (dict(kheads=0), 1), (dict(vheads=3), 1), (dict(dk=0), 1),
             (dict(dv=0), 1), (dict(dtype=7), 1), (dict(scale=float("inf")), 1), (dict(q_stride=(1, -1, 1)), 1),
             (dict(dtype=1), 3), (dict(dv=65537), 3), (dict(batch=(1 << 24) + 1), 3), (dict(tokens=1 << 31), 3)]


@pytest.mark.parametrize("change,status", BAD_SIZES + [(dict(dk=129), 3)])
def test_delta_rule_refuses_sizes(fg, change, status):
    assert forward(fg, desc(fg, **change)) == status
    assert backward(fg, desc(fg, **change)) == status
    assert fg.fft_delta_rule_workspace_bytes(desc(fg, **change), 0) == 0
    assert fg.fft_delta_rule_backward_workspace_bytes(desc(fg, **change), 0) == 0


@pytest.mark.parametrize("change,status", BAD_SIZES + [(dict(dk=257), 3)])
def test_delta_step_refuses_sizes(fg, change, status):
    assert step(fg, desc(fg, **change), pool=1 << 30) == status


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "o", "ws"])
def test_delta_rule_refuses_missing_and_misaligned(fg, name):
    assert forward(fg, desc(fg), **{name: None}) == fg.FFT_ERR_INVALID_ARG
    assert forward(fg, desc(fg), **{name: P + 2}) == fg.FFT_ERR_MISALIGNED


@pytest.mark.parametrize("name", ["do", "q", "k", "v", "g", "beta", "dq", "dk", "dv", "dg", "db", "ws"])
def test_delta_backward_refuses_missing_and_misaligned(fg, name):
    assert backward(fg, desc(fg), **{name: None}) == fg.FFT_ERR_INVALID_ARG
    assert backward(fg, desc(fg), **{name: P + 2}) == fg.FFT_ERR_MISALIGNED


@pytest.mark.parametrize("name", ["s0", "s1", "offsets"])
def test_delta_rule_refuses_misaligned_states(fg, name):
    assert forward(fg, desc(fg), **{name: P + 2}) == fg.FFT_ERR_MISALIGNED


def test_delta_workspaces(fg):
    d = desc(fg)
    need = fg.fft_delta_rule_workspace_bytes(d, 0)
    assert need > 0 and forward(fg, d, nbytes=need - 1) == fg.FFT_ERR_INVALID_ARG
    need = fg.fft_delta_rule_backward_workspace_bytes(d, 1)
    assert need > fg.fft_delta_rule_workspace_bytes(d, 1)
    assert backward(fg, d, offsets=P, nbytes=need - 1) == fg.FFT_ERR_INVALID_ARG
    # packed rows: a partial chunk for every sequence is provided for
    assert fg.fft_delta_rule_workspace_bytes(d, 1) >= fg.fft_delta_rule_workspace_bytes(desc(fg, batch=1, tokens=10), 0)


def test_delta_step_refuses(fg):
    d = desc(fg)
    assert step(fg, d, pool=1) == fg.FFT_ERR_INVALID_ARG       # two sequences, one state
    assert step(fg, d, pool=-1, slots=P) == fg.FFT_ERR_INVALID_ARG
    assert step(fg, d, o=None) == fg.FFT_ERR_INVALID_ARG
    assert step(fg, d, state=None) == fg.FFT_ERR_INVALID_ARG
    assert step(fg, d, slots=P + 2) == fg.FFT_ERR_MISALIGNED
    assert fg._lib.fft_delta_rule_step(None, P, P, P, P, P, P, None, 2, P, None) == fg.FFT_ERR_INVALID_ARG


def test_delta_of_nothing(fg):
    assert forward(fg, desc(fg, batch=0), q=None, o=None, ws=None, nbytes=0) == fg.FFT_OK
    assert backward(fg, desc(fg, batch=0), do=None, ws=None, nbytes=0) == fg.FFT_OK
    assert step(fg, desc(fg, batch=0), q=None, o=None) == fg.FFT_OK
    assert step(fg, desc(fg, tokens=0), q=None, o=None) == fg.FFT_OK
