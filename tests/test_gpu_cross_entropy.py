"""GPU cross entropy of a linear layer and its gradients against the formulas
in 64 bits.

Tolerances, fixed before the first run, per element.  Logits: products of 16-bit
operands are exact, their sum of dim terms in float loses at most 2^-23 of the
sizes summed per addition; float operands lose 2^-24 of each product more by the
parts left out: e_l = (dim + 8) 2^-23 |x| . |w|.  lse and loss are off by the largest
of their token's e_l, 2^-24 of the logits' largest size and 2^-21 (exponentials
of 2^-22, summed) more; and 4 * 2^-24 of lse, which is up to log V above the logits'
size: the logarithm, its sum with the power of two, their product with ln 2 and that
constant round by 2^-24 of it each.  G is off by (2 e_l + 2^-21 + 2^-22 |l - lse|) of
e^{l - lse} c, is then rounded to the operands' type (float: three parts, 2^-24), and
the two products add the sizes |G| |w| with 2^-23 per addition of rounding, before the
results are rounded once.  In half, G has a power of two that brings the largest c to
2^14 .. 2^15, so what is lost below its smallest step is 2^-25 2^-14 of that c.
Float and bfloat16 end at 2^-126: an exponential or a part of G below that may be
taken as 0, so each G may lose 4 * 2^-126 besides.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def inputs(seed, tokens, vocabulary, dim, kind, padded=True, lean=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    w = 2 * dim ** -0.5 * torch.randn(vocabulary, dim, generator=gen, device="cuda")
    targets = torch.from_numpy(rng.integers(vocabulary, size=tokens)).cuda()
    x = torch.randn(tokens, dim, generator=gen, device="cuda")
    x += lean * torch.rand(tokens, 1, generator=gen, device="cuda") * w[targets]
    if padded and tokens > 2:
        bad = torch.from_numpy(rng.random(tokens) < 0.2).cuda()
        targets[bad] = torch.from_numpy(rng.choice([-100, -1, vocabulary, 2 ** 31 - 1], tokens)).cuda()[bad]
    dloss = (0.5 + torch.rand(tokens, generator=gen, device="cuda")) / tokens
    return x.to(TYPES[kind]), w.to(TYPES[kind]), targets, dloss


def check(fg, x, w, targets, dloss, forward_only=False):
    kind, dim = x.dtype, x.shape[-1]
    step = torch.finfo(kind).eps / 2
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    assert loss.dtype == lse.dtype == torch.float32 and loss.shape == targets.shape
    x64, w64 = x.double(), w.double()
    logits = x64 @ w64.t()
    # by columns, to hold one matrix of sizes at a time
    el = (dim + 8) * 2.0 ** -23 * (x64.abs() @ w64.abs().t())
    want = torch.logsumexp(logits, 1)
    there = (targets >= 0) & (targets < w.shape[0])
    at = torch.where(there, targets, 0)[:, None]
    tol = el.amax(1) + 2.0 ** -23 * logits.abs().amax(1) + 2.0 ** -21 + 2.0 ** -22 * want.abs()
    assert ((lse.double() - want).abs() <= tol).all()
    want_loss = torch.where(there, want - logits.gather(1, at)[:, 0], 0)
    assert ((loss.double() - want_loss).abs() <= 2 * tol).all()
    assert not loss[~there].any()
    again = fg.linear_cross_entropy(x, w, targets)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
    if forward_only:
        return
    dx, dw = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    c = torch.where(there, dloss.double(), 0)[:, None]
    # from the lse that the call was given
    p = (logits - lse.double()[:, None]).exp()
    rel = 2 * el + 2.0 ** -21 + 2.0 ** -22 * (logits - lse.double()[:, None]).abs()
    err = p * rel
    G = p.scatter_add(1, at, -torch.ones_like(at, dtype=torch.float64)) * c
    err = err * c.abs() + G.abs() * (step if kind != torch.float32 else 2.0 ** -23)
    if kind == torch.float16:
        err = err + 2.0 ** -39 * dloss.abs().max() * 2
    err = err + 2.0 ** -124
    err = torch.where(there[:, None], err, 0)
    for got, left, right, e in ((dx, G, w64, err), (dw, G.t(), x64, err.t())):
        exact, size, lost = left @ right, left.abs() @ right.abs(), e @ right.abs()
        bound = step * exact.abs() + (lost + (left.shape[1] + 16) * 2.0 ** -23 * size) * (1 + step)
        if kind == torch.float16:
            bound = bound + 2.0 ** -25
        bad = ~((got.double() - exact).abs() <= bound + 1e-300)
        assert got.dtype == kind and not bad.any(), \
            f"{int(bad.sum())} of {bad.numel()}, worst {float(((got.double() - exact).abs() / bound).max())}"
    one, other = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert torch.equal(one, dx) and torch.equal(other, dw)


SHAPES = [(1, 1, 1), (1, 2, 8), (5, 3, 7), (2, 127, 16), (3, 128, 63), (48, 129, 64), (33, 255, 65), (127, 256, 200),
          (128, 257, 128), (129, 1000, 40), (256, 300, 512), (257, 2049, 72), (700, 777, 333), (30, 9000, 96)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens,vocabulary,dim", SHAPES)
def test_loss_and_gradients(fg, tokens, vocabulary, dim, kind):
    check(fg, *inputs(tokens + dim, tokens, vocabulary, dim, kind))


@pytest.mark.parametrize("kind", list(TYPES))
def test_many_tiles(fg, kind):
    check(fg, *inputs(1, 1500, 20001, 264, kind))


@pytest.mark.parametrize("kind,tokens,vocabulary,dim", [("f32", 40000, 2500, 40), ("bf16", 60000, 5000, 24),
                                                        ("f16", 60000, 4353, 8)])
def test_pieces_of_the_vocabulary(fg, kind, tokens, vocabulary, dim):
    check(fg, *inputs(2, tokens, vocabulary, dim, kind))


@pytest.mark.parametrize("kind,tokens,vocabulary,dim", [("f16", 30000, 300, 72), ("bf16", 40000, 257, 33),
                                                        ("f32", 20000, 90, 100), ("bf16", 9000, 256, 520)])
def test_few_words_for_many_tokens(fg, kind, tokens, vocabulary, dim):
    check(fg, *inputs(17, tokens, vocabulary, dim, kind))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_operands_off_their_boundaries(fg, kind):
    x, w, targets, dloss = inputs(3, 90, 400, 64, kind)
    want = fg.linear_cross_entropy(x, w, targets)
    grads = fg.linear_cross_entropy_backward(dloss, x, w, targets, want[1])

    def padded(t):
        wide = torch.full((t.shape[0], t.shape[1] + 9), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, 3:3 + t.shape[1]] = t
        return wide[:, 3:3 + t.shape[1]]

    def spaced(t):
        wide = torch.full((t.shape[0], 2 * t.shape[1]), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, :t.shape[1]] = t
        return wide[:, :t.shape[1]]
    for f in (padded, spaced, lambda t: t.t().contiguous().t()):
        got = fg.linear_cross_entropy(f(x), f(w), targets.int())
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        got = fg.linear_cross_entropy_backward(dloss, f(x), f(w), targets.int(), want[1])
        assert all(torch.equal(p, q) for p, q in zip(got, grads))


def test_shapes_and_parts_of_the_gradient(fg):
    x, w, targets, dloss = inputs(4, 60, 90, 32, "bf16")
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    three = lambda t: t.reshape(3, 20, *t.shape[1:])  # noqa: E731
    l3, s3 = fg.linear_cross_entropy(three(x), w, three(targets))
    assert torch.equal(l3, three(loss)) and torch.equal(s3, three(lse))
    dx, dw = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    d3, w3 = fg.linear_cross_entropy_backward(three(dloss), three(x), w, three(targets), s3)
    assert torch.equal(d3, three(dx)) and torch.equal(w3, dw)
    only, none = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dweight=False)
    assert none is None and torch.equal(only, dx)
    none, only = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse, dx=False)
    assert none is None and torch.equal(only, dw)
    mean = torch.ones((), device="cuda").div(60).expand(60)
    check(fg, x, w, targets, mean)


@pytest.mark.parametrize("kind", list(TYPES))
def test_tokens_without_a_target_may_hold_anything(fg, kind):
    x, w, targets, dloss = inputs(5, 300, 500, 72, kind)
    none = targets < 0
    none[7] = True
    targets[7] = -100
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    dx, dw = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    for junk in (float("nan"), float("inf"), -torch.finfo(TYPES[kind]).max):
        y = x.clone()
        y[none] = junk
        l2, s2 = fg.linear_cross_entropy(y, w, targets)
        assert torch.equal(l2, loss) and torch.equal(s2[~none], lse[~none])
        s2[none] = float("nan")
        e2, f2 = fg.linear_cross_entropy_backward(dloss, y, w, targets, s2)
        assert torch.equal(e2, dx) and torch.equal(f2, dw) and not e2[none].any()
    # no target at all
    targets[:] = -1
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    dx, dw = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    assert not loss.any() and not dx.any() and not dw.any()


def test_words_that_cannot_be(fg):
    # logits of -infinity in whole tiles: weight 0, the others as without them
    x, w, targets, dloss = inputs(6, 50, 700, 64, "bf16", padded=False)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    small, s = w[:130].contiguous(), targets % 130
    loss, lse = fg.linear_cross_entropy(x, small, s)
    w[130:] = 0
    w[130:, 0] = -float("inf")
    x[:, 1:] = x[:, 1:].abs() + 0.5  # no 0 times infinity
    loss, lse = fg.linear_cross_entropy(x, small, s)
    l2, s2 = fg.linear_cross_entropy(x, w, s)
    assert torch.equal(l2, loss) and torch.equal(s2, lse)


@pytest.mark.parametrize("kind", list(TYPES))
def test_words_masked_by_the_lowest_value(fg, kind):
    # logits at the end of the type's range, alone in their tiles and between others
    x, w, targets, dloss = inputs(16, 60, 700, 64, kind, padded=False)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    targets %= 130
    loss, lse = fg.linear_cross_entropy(x, w[:130].contiguous(), targets)
    grads = fg.linear_cross_entropy_backward(dloss, x, w[:130].contiguous(), targets, lse)
    w[130:] = 0
    w[130:, 0] = torch.finfo(TYPES[kind]).min
    order = torch.randperm(700, device="cuda")
    back = torch.argsort(order)
    for words, t in ((w, targets), (w[order], back[targets])):
        l2, s2 = fg.linear_cross_entropy(x, words, t)
        # the sums of another order of words
        assert ((l2 - loss).abs() <= 1e-5 * (1 + loss.abs())).all() and ((s2 - lse).abs() <= 1e-5 * (1 + lse.abs())).all()
        dx, dw = fg.linear_cross_entropy_backward(dloss, x, words, t, s2)
        step = torch.finfo(TYPES[kind]).eps
        assert ((dx.double() - grads[0].double()).abs() <= 2 * step * grads[0].double().abs().max() + 1e-7).all()
        dw = dw[back] if t is not targets else dw
        assert not dw[130:].any()
        assert ((dw[:130].double() - grads[1].double()).abs() <= 2 * step * grads[1].double().abs().max() + 1e-7).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_large_logits(fg, kind):
    x, w, targets, dloss = inputs(7, 40, 300, 64, kind)
    check(fg, (x * 30).to(x.dtype), w, targets, dloss)


def test_small_weights_of_half(fg):
    # dloss far below half's smallest value: G is scaled
    x, w, targets, dloss = inputs(8, 64, 200, 64, "f16")
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    big = fg.linear_cross_entropy_backward(dloss * 2.0 ** 5, x, w, targets, lse)[0].double()
    small = fg.linear_cross_entropy_backward(dloss * 2.0 ** -3, x, w, targets, lse)[0].double()
    assert ((small * 2.0 ** 8 - big).abs() <= 2.0 ** -25 * 2.0 ** 8).all()


def test_gradient_against_differences(fg):
    x, w, targets, dloss = inputs(9, 20, 50, 24, "f32")
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    dx, dw = fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    vx, vw = torch.randn_like(x, dtype=torch.float64), torch.randn_like(w, dtype=torch.float64)
    there = targets >= 0
    there &= targets < 50

    def value(e):
        logits = (x.double() + e * vx) @ (w.double() + e * vw).t()
        each = torch.logsumexp(logits, 1) - logits.gather(1, torch.where(there, targets, 0)[:, None])[:, 0]
        return float((each * dloss.double() * there).sum())
    h = 1e-4
    want = (value(h) - value(-h)) / (2 * h)
    got = float((dx * vx).sum() + (dw * vw).sum())
    assert abs(got - want) <= 1e-5 * float((dx * vx).abs().sum() + (dw * vw).abs().sum())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_long_sums_of_one_sign(fg, kind):
    # An addition of 16 terms on the tensor cores may cut off 2^-23 of the sum so far: 32 of them in 512
    # terms (float: six products of parts, of which only one is not small), then sums rounded to nearest.
    bound = lambda terms: 40 * 2.0 ** -23 + (terms / 512 + 8) * 2.0 ** -24  # noqa: E731
    x = torch.rand(70, 16384, device="cuda").to(TYPES[kind])
    w = (torch.rand(1, 16384, device="cuda") / 16384).to(TYPES[kind])
    lse = fg.linear_cross_entropy(x, w, torch.zeros(70, dtype=torch.int64, device="cuda"))[1]
    want = (x.double() @ w.double().t())[:, 0]
    assert ((lse.double() / want - 1).abs() <= bound(16384)).all()
    # dw over tokens: two words of equal weight, all targets the first
    x = torch.rand(20000, 40, device="cuda").to(TYPES[kind])
    w, targets = torch.zeros(2, 40, device="cuda").to(TYPES[kind]), torch.zeros(20000, dtype=torch.int64, device="cuda")
    dloss = torch.full((20000,), 2.0 ** -10, device="cuda")
    dw = fg.linear_cross_entropy_backward(dloss, x, w, targets, fg.linear_cross_entropy(x, w, targets)[1])[1]
    want = 2.0 ** -11 * x.double().sum(0)
    step = torch.finfo(TYPES[kind]).eps / 2 if kind != "f32" else 0
    assert ((dw[1].double() / want - 1).abs() <= bound(20000) + 2.0 ** -20 + step).all()
    # dx over words: equal logits of 0, the target's weights 0, the others positive
    w = torch.rand(30000, 40, device="cuda").to(TYPES[kind])
    w[0] = 0
    x = torch.zeros(9, 40, device="cuda").to(TYPES[kind])
    targets = torch.zeros(9, dtype=torch.int64, device="cuda")
    lse = fg.linear_cross_entropy(x, w, targets)[1]
    dx = fg.linear_cross_entropy_backward(torch.ones(9, device="cuda"), x, w, targets, lse)[0]
    p = torch.exp(-lse.double())[:, None]
    if kind == "bf16":  # one rounding of every p alike
        p = p.to(TYPES[kind]).double()
    assert ((dx.double() / (p * w.double().sum(0)) - 1).abs() <= bound(30000) + 2.0 ** -20 + step).all()


def test_nothing_and_refusals(fg):
    x, w, targets, dloss = inputs(10, 10, 20, 16, "f32")
    loss, lse = fg.linear_cross_entropy(x[:0], w, targets[:0])
    assert loss.shape == (0,)
    junk = torch.full((320,), float("nan"), device="cuda")
    del junk
    dx, dw = fg.linear_cross_entropy_backward(dloss[:0], x[:0], w, targets[:0], lse)
    assert dx.shape == (0, 16) and not dw.any()
    loss, lse = fg.linear_cross_entropy(x, w, targets)
    for bad in (lambda: fg.linear_cross_entropy(x[:, :8], w, targets), lambda: fg.linear_cross_entropy(x, w, targets[:5]),
                lambda: fg.linear_cross_entropy(x, w[0], targets), lambda: fg.linear_cross_entropy(x.cpu(), w, targets),
                lambda: fg.linear_cross_entropy_backward(dloss.double(), x, w, targets, lse),
                lambda: fg.linear_cross_entropy_backward(dloss, x, w, targets, lse[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fg.linear_cross_entropy(x, w.bfloat16(), targets)
    with pytest.raises(TypeError):
        fg.linear_cross_entropy(x, w, targets.float())
    with pytest.raises(fg.FFTError):
        fg.linear_cross_entropy(x.double(), w.double(), targets)


@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_captured_and_replayed(fg, kind):
    x, w, targets, dloss = inputs(11, 200, 600, 80, kind)
    stream = torch.cuda.Stream()

    def run():
        loss, lse = fg.linear_cross_entropy(x, w, targets)
        return loss, lse, *fg.linear_cross_entropy_backward(dloss, x, w, targets, lse)
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in (12, 13):
        for t, n in zip((x, w, targets, dloss), inputs(seed, 200, 600, 80, kind)):
            t.copy_(n)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(got, run()))


def test_two_streams_at_once(fg):
    a, b = inputs(14, 300, 3000, 128, "bf16"), inputs(15, 400, 2000, 136, "f32")
    want = [fg.linear_cross_entropy(*t[:3]) for t in (a, b)]
    grads = [fg.linear_cross_entropy_backward(t[3], *t[:3], s[1]) for t, s in zip((a, b), want)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [fg.linear_cross_entropy_backward(t[3], *t[:3], s[1], stream=st) for t, s, st in zip((a, b), want, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for x, y in zip(got, grads) for p, q in zip(x, y))
    assert fg.fft_device_status(None) == fg.FFT_OK
