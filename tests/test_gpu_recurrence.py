"""GPU gated linear recurrence, its gradients and single tokens against the
recurrence in 64 bits.

Tolerances, fixed before the first run, per element: a result is rounded once
to its type.  Before that, state t is a sum of terms e^{g_t + .. + g_{j+1}} b_j x_j;
a factor's exponential is off by 2 units of 2^-23 at most, its product and the sum
by half a unit each, and the maps that carry states over warps and blocks by
two more products: 6 * 2^-24 per step that a term has gone and 16 * 2^-24 at its
ends.  With S_t the sum of the terms' sizes and N_t that of sizes times steps (both
follow the same recurrence, in 64 bits) that is (16 S + 6 N) 2^-24.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def half_step(kind):
    return torch.finfo(kind).eps / 2


def tiny(kind):
    return 2.0 ** -25 if kind == torch.float16 else 2.0 ** -140


def inputs(seed, shape, kind, gkind, gated=True, initial=None):
    rng = np.random.default_rng(seed)
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s)).cuda()  # noqa: E731
    rate = torch.logspace(-3, 0.7, shape[-1], dtype=torch.float64, device="cuda")
    x = normal(*shape).to(kind)
    g = (-rate * torch.nn.functional.softplus(normal(*shape))).to(gkind)
    beta = torch.sigmoid(normal(*shape)).to(gkind) if gated else None
    h0 = normal(initial, shape[-1]).float() if initial else None
    return x, g, beta, h0, normal(*shape).to(kind), normal(*(initial or 1, shape[-1])).float()


def bounds_of(lengths, packed, tokens):
    if packed is None:
        return [(slice(i, i + 1), 0, tokens) for i in range(lengths)]
    out, low = [], 0
    ends = [min(max(v, 0), tokens) for v in packed]
    for i in range(len(ends)):
        low = max(low, ends[i])
        ends[i] = low
    return [(None, a, b) for a, b in zip(ends[:-1], ends[1:])]


def rows_of(t, seq):
    """The rows [tokens of the sequence, channels] of a batch or a packed array."""
    s, a, b = seq
    return t[a:b] if s is None else t[s][0, a:b]


def forward64(x, g, beta, h):
    """y, the sums of sizes S and of sizes times steps N, per token; and the three behind the last."""
    x, a = x.double(), g.double().exp()
    u = x if beta is None else x * beta.double()
    h = u.new_zeros(u.shape[1:]) if h is None else h.double()
    s, n = h.abs(), torch.zeros_like(h)
    rows = []
    for t in range(len(u)):
        h, n = a[t] * h + u[t], a[t] * (n + s)
        s = a[t] * s + u[t].abs()
        rows.append((h, s, n))
    return [torch.stack(r) for r in zip(*rows)] if rows else [u] * 3, (h, s, n)


def backward64(dy, x, g, y, beta, h0, d):
    x, a, dy, y = x.double(), g.double().exp(), dy.double(), y.double()
    b = torch.ones_like(x) if beta is None else beta.double()
    d = x.new_zeros(x.shape[1:]) if d is None else d.double()
    s, n = d.abs(), torch.zeros_like(d)
    h0 = torch.zeros_like(d) if h0 is None else h0.double()
    rows = [None] * len(x)
    for t in reversed(range(len(x))):
        before = y[t - 1] if t else h0
        d, s = d + dy[t], s + dy[t].abs()
        size = U * (16 * s + 6 * n)
        rows[t] = (b[t] * d, b[t] * size, a[t] * d * before, a[t] * size * before.abs() + 8 * U * (a[t] * d * before).abs(),
                   x[t] * d, x[t].abs() * size)
        d, n, s = a[t] * d, a[t] * (n + s), a[t] * s
    return [torch.stack(r) for r in zip(*rows)] if rows else None, (d, U * (16 * s + 6 * n))


def within(got, want, size):
    kind = got.dtype
    bound = half_step(kind) * want.abs() + size * (1 + half_step(kind)) + tiny(kind)
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {float(((got.double() - want).abs() / bound).max())}"


def check(fg, args, seqs, offsets=None, dfinal=True):
    x, g, beta, h0, dy, d1 = args
    y, final = fg.linear_recurrence(x, g, beta, initial_state=h0, offsets=offsets)
    again = fg.linear_recurrence(x, g, beta, initial_state=h0, offsets=offsets)
    assert torch.equal(y, again[0]) and torch.equal(final, again[1])
    d1 = torch.randn(final.shape, device="cuda") if dfinal else None
    dx, dg, db, d0 = fg.linear_recurrence_backward(dy, x, g, y, beta=beta, initial_state=h0, offsets=offsets,
                                                   dfinal_state=d1)
    assert (db is None) == (beta is None) and dg.dtype == g.dtype and dx.dtype == x.dtype
    for i, seq in enumerate(seqs):
        r = lambda t: None if t is None else rows_of(t, seq)  # noqa: E731
        start = None if h0 is None else h0[i]
        (want, s, n), end = forward64(r(x), r(g), r(beta), start)
        if len(want):
            within(r(y), want, U * (16 * s + 6 * n))
        within(final[i], end[0], U * (16 * end[1] + 6 * end[2]))
        rows, last = backward64(r(dy), r(x), r(g), r(y), r(beta), start, None if d1 is None else d1[i])
        within(d0[i], last[0], last[1])
        if rows is None:
            continue
        within(r(dx), rows[0], rows[1] + 4 * U * rows[0].abs())
        within(r(dg), rows[2], rows[3])
        if beta is not None:
            within(r(db), rows[4], rows[5] + 4 * U * rows[4].abs())


KINDS = [("f32", "f32", True), ("f32", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", False), ("f16", "f32", True),
         ("f16", "f16", False)]


@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("batch,tokens,channels", [(1, 1, 1), (2, 3, 5), (1, 4, 128), (3, 33, 132), (2, 257, 64), (1, 300, 7),
                                                   (1, 1025, 260), (40, 70, 516), (5, 500, 1024), (1, 2500, 130)])
def test_batches(fg, batch, tokens, channels, kind, gkind, gated):
    args = inputs(batch + tokens, (batch, tokens, channels), TYPES[kind], TYPES[gkind], gated, batch)
    check(fg, args, bounds_of(batch, None, tokens))


@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("offsets", [[0, 1, 1, 40, 200], [0, 200], [0] * 3 + [200], [10, 70, 70, 150], [0, 130], [200], [0, 0, 0],
                                     [0, 90, 40, 210, 100], [-5, 50, 2 ** 30]])
@pytest.mark.parametrize("channels", [40, 129])
def test_packed(fg, channels, offsets, kind, gkind, gated):
    n = len(offsets) - 1
    args = inputs(7, (200, channels), TYPES[kind], TYPES[gkind], gated, None)
    x, g, beta, _, dy, _ = args
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    h0 = torch.randn(n, channels, device="cuda") if n else None
    seqs = bounds_of(n, offsets, 200)
    junk = [torch.full((200 * channels,), float("nan"), device="cuda") for _ in range(4)]
    del junk
    check(fg, (x, g, beta, h0, dy, None), seqs, at)
    check(fg, (x, g, beta, None, dy, None), seqs, at, dfinal=False)
    # rows of no sequence: 0 in new results, untouched in those that are given
    y, _ = fg.linear_recurrence(x, g, beta, offsets=at)
    kept = torch.full_like(y, 3.0)
    fg.linear_recurrence(x, g, beta, offsets=at, out=kept)
    grads = fg.linear_recurrence_backward(dy, x, g, y, beta=beta, offsets=at)[:3]
    used = torch.zeros(200, dtype=torch.bool, device="cuda")
    for _, a, b in seqs:
        used[a:b] = True
    assert torch.equal(kept[used], y[used]) and (kept[~used] == 3).all()
    for t in (y, *grads):
        assert t is None or (not t[~used].any() and t.isfinite().all())


@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("channels", [136, 45])
def test_long_packed(fg, channels, kind, gkind, gated):
    # sequences of different lengths of several steps, and rows of none on both sides
    offsets = [5, 700, 701, 701, 1990]
    x, g, beta, _, dy, _ = inputs(13, (2000, channels), TYPES[kind], TYPES[gkind], gated)
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    h0 = torch.randn(4, channels, device="cuda")
    check(fg, (x, g, beta, h0, dy, None), bounds_of(4, offsets, 2000), at)
    y, _ = fg.linear_recurrence(x, g, beta, offsets=at)
    assert not y[:5].any() and not y[1990:].any()


@pytest.mark.parametrize("sequences", [1024, 1025, 3000])
def test_many_packed_sequences(fg, sequences):
    rng = np.random.default_rng(sequences)
    lengths = rng.integers(0, 4, sequences)
    ends = np.concatenate([[3], 3 + np.cumsum(lengths)])
    tokens = int(ends[-1]) + 2
    x, g, beta, _, dy, _ = inputs(12, (tokens, 36), torch.bfloat16, torch.float32, True)
    h0 = torch.randn(sequences, 36, device="cuda")
    at = torch.tensor(ends, dtype=torch.int32, device="cuda")
    y, final = fg.linear_recurrence(x, g, beta, initial_state=h0, offsets=at)
    dx, dg, db, d0 = fg.linear_recurrence_backward(dy, x, g, y, beta=beta, initial_state=h0, offsets=at)
    for t in (y, dx, dg, db):
        assert not t[:3].any() and not t[-2:].any()
    for i in rng.choice(sequences, 60, replace=False):
        a, b = int(ends[i]), int(ends[i + 1])
        (want, s, n), end = forward64(x[a:b], g[a:b], beta[a:b], h0[i])
        within(final[i], end[0], U * (16 * end[1] + 6 * end[2]))
        rows, last = backward64(dy[a:b], x[a:b], g[a:b], y[a:b], beta[a:b], h0[i], None)
        within(d0[i], last[0], last[1])
        if b > a:
            within(y[a:b], want, U * (16 * s + 6 * n))
            within(dx[a:b], rows[0], rows[1] + 4 * U * rows[0].abs())
            within(dg[a:b], rows[2], rows[3])
            within(db[a:b], rows[4], rows[5] + 4 * U * rows[4].abs())


def test_clusters_agree_with_parts(fg):
    # one long sequence (blocks of a cluster share its tokens) against its pieces with carried states
    x, g, beta, h0, _, _ = inputs(3, (1, 4000, 96), torch.float32, torch.float32, True, 1)
    y, final = fg.linear_recurrence(x, g, beta, initial_state=h0)
    (want, s, n), end = forward64(x[0], g[0], beta[0], h0[0])
    within(y[0], want, U * (16 * s + 6 * n))
    state, parts = h0, []
    for a, b in ((0, 1), (1, 900), (900, 901), (901, 4000)):
        part, state = fg.linear_recurrence(x[:, a:b], g[:, a:b], beta[:, a:b], initial_state=state)
        parts.append(part)
    within(torch.cat(parts, 1)[0], want, U * (16 * s + 6 * n))
    within(state[0], end[0], U * (16 * end[1] + 6 * end[2]))


def test_decays_that_drop_or_grow(fg):
    x, g, beta, h0, dy, _ = inputs(4, (2, 150, 33), torch.float32, torch.float32, True, 2)
    g[:, 60] = -float("inf")
    g[:, 100:110] = -200.0
    check(fg, (x, g, beta, h0, dy, None), bounds_of(2, None, 150))
    # growth: products of decays overflow where the state is still 0
    g = torch.full((1, 64, 8), 30.0, device="cuda")
    x = torch.zeros(1, 64, 8, device="cuda")
    x[:, 62] = 1.0
    y, final = fg.linear_recurrence(x, g)
    assert not y[:, :62].any() and (y[:, 62] == 1).all() and final.isfinite().all()


def test_what_is_not_finite_stays_where_it_is(fg):
    x, g, beta, h0, _, _ = inputs(5, (1, 300, 64), torch.float32, torch.float32, True, 1)
    clean, _ = fg.linear_recurrence(x, g, beta, initial_state=h0)
    x[0, 130, 5] = float("nan")
    x[0, 200, 9] = float("inf")
    y, _ = fg.linear_recurrence(x, g, beta, initial_state=h0)
    other = [c for c in range(64) if c not in (5, 9)]
    assert torch.equal(y[..., other], clean[..., other])
    assert torch.equal(y[0, :130, 5], clean[0, :130, 5]) and y[0, 130:, 5].isnan().all()
    assert torch.equal(y[0, :200, 9], clean[0, :200, 9])


def test_strides(fg):
    base = torch.randn(3, 50, 3, 72, device="cuda")
    x, g, beta = base[:, :, 0], -base[:, :, 1].abs(), torch.sigmoid(base)[:, :, 2]
    want = fg.linear_recurrence(x.contiguous(), g.contiguous(), beta.contiguous())
    dy = torch.randn(3, 50, 72, device="cuda")
    grads = fg.linear_recurrence_backward(dy, x.contiguous(), g.contiguous(), want[0], beta=beta.contiguous())
    for f in (lambda t: t, lambda t: t.transpose(0, 1).contiguous().transpose(0, 1),
              lambda t: torch.cat([t.new_zeros(3, 50, 1), t], 2)[..., 1:], lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)):
        got = fg.linear_recurrence(f(x), f(g), f(beta))
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        got = fg.linear_recurrence_backward(f(dy), f(x), f(g), f(want[0]), beta=f(beta))
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
    # one decay for all tokens and sequences, expanded
    one = g[:1, :1].expand(3, 50, 72)
    assert torch.equal(fg.linear_recurrence(x, one)[0], fg.linear_recurrence(x, one.contiguous())[0])


@pytest.mark.parametrize("kind,gkind,gated", KINDS)
@pytest.mark.parametrize("batch,tokens,channels", [(1, 1, 1), (3, 1, 128), (5, 4, 260), (70, 2, 33), (9, 1, 1030)])
def test_single_tokens(fg, batch, tokens, channels, kind, gkind, gated):
    x, g, beta, _, _, _ = inputs(6, (batch, tokens, channels), TYPES[kind], TYPES[gkind], gated)
    pool = torch.randn(2 * batch + 3, channels, device="cuda")
    slots = torch.randperm(2 * batch + 3, device="cuda")[:batch].int()
    if batch > 2:
        slots[1] = -1
        slots[2] = 2 * batch + 3
    before = pool.clone()
    y = fg.linear_recurrence_step(x, g, pool, beta=beta, slots=slots)
    named = torch.zeros(len(pool), dtype=torch.bool, device="cuda")
    for i, s in enumerate(slots.tolist()):
        if not 0 <= s < len(pool):
            assert not y[i].any()
            continue
        named[s] = True
        (want, size, n), end = forward64(x[i], g[i], None if beta is None else beta[i], before[s])
        within(y[i], want, U * (16 * size + 6 * n))
        within(pool[s], end[0], U * (16 * end[1] + 6 * end[2]))
    assert torch.equal(pool[~named], before[~named])


def test_decoding_continues_a_prompt(fg):
    x, g, beta, _, _, _ = inputs(8, (4, 40, 100), torch.bfloat16, torch.float32, True)
    y, final = fg.linear_recurrence(x, g, beta)
    state = fg.linear_recurrence(x[:, :30], g[:, :30], beta[:, :30])[1]
    for t in range(30, 40):
        one = fg.linear_recurrence_step(x[:, t:t + 1], g[:, t:t + 1], state, beta=beta[:, t:t + 1])
        assert (one[:, 0].float() - y[:, t].float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()
    assert (state - final).abs().max() <= 1e-5 * final.abs().max()


def test_gradients_against_differences(fg):
    # central differences of the 64-bit recurrence along a random direction: h^2 of curvature
    x, g, beta, h0, dy, _ = inputs(9, (1, 30, 12), torch.float32, torch.float32, True, 1)
    d1 = torch.randn(1, 12, device="cuda")
    y, _ = fg.linear_recurrence(x, g, beta, initial_state=h0)
    grads = fg.linear_recurrence_backward(dy, x, g, y, beta=beta, initial_state=h0, dfinal_state=d1)
    dirs = [torch.randn_like(t, dtype=torch.float64) for t in (x, g, beta, h0)]

    def value(e):
        p = [t.double() + e * d for t, d in zip((x, g, beta, h0), dirs)]
        (out, _, _), end = forward64(p[0][0], p[1][0], p[2][0], p[3][0])
        return (out * dy[0].double()).sum() + (end[0] * d1[0].double()).sum()
    h = 1e-4
    want = float(value(h) - value(-h)) / (2 * h)
    got = sum(float((a.double() * b).sum()) for a, b in zip(grads, dirs))
    size = sum(float((a.double() * b).abs().sum()) for a, b in zip(grads, dirs))
    assert abs(got - want) <= 1e-5 * size


def test_states_in_place_and_refusals(fg):
    x, g, beta, h0, dy, _ = inputs(10, (2, 20, 48), torch.float32, torch.float32, True, 2)
    with pytest.raises(ValueError):
        fg.linear_recurrence(x, g[:, :5], beta)
    with pytest.raises(ValueError):
        fg.linear_recurrence(x[0], g[0], beta[0])
    with pytest.raises(TypeError):
        fg.linear_recurrence(x, g.bfloat16())
    with pytest.raises(TypeError):
        fg.linear_recurrence(x.bfloat16(), g, beta.bfloat16())
    with pytest.raises(fg.FFTError):
        fg.linear_recurrence(x.double(), g.double())
    with pytest.raises(ValueError):
        fg.linear_recurrence(x, g, initial_state=h0[:1])
    with pytest.raises(ValueError):
        fg.linear_recurrence_backward(dy[:, :3], x, g, x)
    with pytest.raises(ValueError):
        fg.linear_recurrence_step(x, g, torch.zeros(2, 47, device="cuda"))
    with pytest.raises(fg.FFTError):
        fg.linear_recurrence_step(x, g, torch.zeros(1, 48, device="cuda"))


def test_captured_and_replayed(fg):
    x, g, beta, h0, dy, _ = inputs(11, (2, 600, 64), torch.bfloat16, torch.bfloat16, True, 2)
    pool = torch.zeros(2, 64, device="cuda")
    stream = torch.cuda.Stream()

    def run():
        y, final = fg.linear_recurrence(x, g, beta, initial_state=h0)
        return y, final, *fg.linear_recurrence_backward(dy, x, g, y, beta=beta, initial_state=h0)
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
        token = fg.linear_recurrence_step(x[:, :1], g[:, :1], pool)
    for seed in (1, 2):
        for t, n in zip((x, g, beta, h0, dy), inputs(seed, (2, 600, 64), torch.bfloat16, torch.bfloat16, True, 2)):
            t.copy_(n)
        pool.zero_()
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(got, run()))
        assert torch.equal(token[:, 0].float(), x[:, 0].float()) and torch.equal(pool, x[:, 0].float())
