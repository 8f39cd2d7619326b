"""Decays above 1 whose products leave float's range, followed by a decay of 0: a
state of 0 stays 0, and what comes behind the drop is not felt before it nor what was
before it behind it.  Against the recurrence in 64 bits, with the bounds of
test_gpu_recurrence.py: where the state is 0 they leave nothing but 2^-140 (half:
2^-25)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_recurrence import KINDS, TYPES, U, backward64, bounds_of, check, forward64, inputs, within  # noqa: E402


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def check_batch(fg, x, g, beta, h0, dy, _):
    """`check` of a batch, all sequences at once."""
    y, final = fg.linear_recurrence(x, g, beta, initial_state=h0)
    d1 = torch.randn_like(final)
    dx, dg, db, d0 = fg.linear_recurrence_backward(dy, x, g, y, beta=beta, initial_state=h0, dfinal_state=d1)
    t = lambda a: None if a is None else a.transpose(0, 1)  # noqa: E731
    (want, s, n), end = forward64(t(x), t(g), t(beta), h0)
    within(t(y), want, U * (16 * s + 6 * n))
    within(final, end[0], U * (16 * end[1] + 6 * end[2]))
    rows, last = backward64(t(dy), t(x), t(g), t(y), t(beta), h0, d1)
    within(d0, last[0], last[1])
    within(t(dx), rows[0], rows[1] + 4 * U * rows[0].abs())
    within(t(dg), rows[2], rows[3])
    if beta is not None:
        within(t(db), rows[4], rows[5] + 4 * U * rows[4].abs())


def with_regions(args, grow):
    """Sequence i has, from token i on, a drop, `grow` decays of e^30, a drop, as many again, and a drop, where neither
    the state (forwards) nor its gradient (backwards) gets anything."""
    x, g, beta, h0, dy, d1 = args
    for i in range(len(x)):
        end = i + 2 * grow + 3
        g[i, i:end] = 30.0
        g[i, [i, i + grow + 1, end - 1]] = -float("inf")
        x[i, i:end] = 0.0
        dy[i, i:end] = 0.0
    return x, g, beta, h0, dy, d1


# within a warp's tokens (at every place of them), across the warps of a block, and across the blocks of a cluster
@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("tokens,grow", [(80, 3), (80, 25), (400, 3), (400, 25), (400, 150), (1500, 600)])
@pytest.mark.parametrize("channels", [8, 13, 1100])  # clusters; copies by lanes; a block per sequence and 128 channels
def test_growth_and_drops(fg, channels, tokens, grow, kind, gkind, gated):
    batch = 2 if tokens > 400 else 18
    args = inputs(tokens + grow, (batch, tokens, channels), TYPES[kind], TYPES[gkind], gated, batch)
    check_batch(fg, *with_regions(args, grow))


@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("channels", [8, 13])
def test_packed_growth_and_drops(fg, channels, kind, gkind, gated):
    x, g, beta, _, dy, _ = with_regions(inputs(5, (1, 900, channels), TYPES[kind], TYPES[gkind], gated), 140)
    flat = [None if t is None else t[0].contiguous() for t in (x, g, beta, dy)]
    # the growth goes on over a border, in front of which the state is 0
    offsets = [0, 60, 61, 200, 900]
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    check(fg, (flat[0], flat[1], flat[2], None, flat[3], None), bounds_of(4, offsets, 900), at, dfinal=False)


@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("tokens", [40, 300])
def test_a_small_state_that_grows_and_is_dropped(fg, tokens, kind, gkind, gated):
    x, g, beta, h0, _, _ = inputs(6, (18, tokens, 8), TYPES[kind], TYPES[gkind], gated, 18)
    x.zero_()
    g.zero_()
    # four steps pass float's range together, three do not (e^87 = 6e37), so that no map of them that hands a state on is cut;
    # halves would not hold what four make of a float
    steps = 2 if kind == "f16" else 4
    h0.fill_(1e-25 if kind == "f16" else 1e-34)
    for i in range(18):
        g[i, i:i + steps] = 29.0
        g[i, i + steps] = -float("inf")
    y, final = fg.linear_recurrence(x, g, beta, initial_state=h0)
    (want, s, _), _ = forward64(*(None if a is None else a.transpose(0, 1) for a in (x, g, beta)), h0)
    # beside the 6 of a step: the exponent 29 log2 e is off by 2^-24 of it and by 0.22 * 2^-24 through the constant,
    # which is 29 * 1.22 * 2^-24 of the decay
    within(y.transpose(0, 1), want, U * (16 + 42 * steps) * s)
    for i in range(18):
        assert not y[i, i + steps:].any()
    assert not final.any()
