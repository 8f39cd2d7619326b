"""GPU gradients of the gated delta rule against the recurrence run backwards
in 64 bits, and that one against differences of the forward recurrence.

Tolerances (relative L2), fixed before the first run: a gradient passes
through at most twelve products one after the other (the forward scan, the
backward one, and the products of both), each keeping 22 significand bits of
every factor and fp32 sums: FP = 12 * 2^-20 = 1.1e-5 for what is returned in
fp32.  dg is a sum over a chunk of differences of such terms: 4 FP.  A
gradient rounded to p bits adds 2^-p.
"""
import pytest

torch = pytest.importorskip("torch")
import delta_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FP = 12 * 2.0 ** -20
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial")


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def run(fg, args, do, state=None, dfinal=None, offsets=None, **more):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    grads = fg.delta_rule_backward(do.cuda(), *cuda(args), initial_state=c(state), dfinal_state=c(dfinal),
                                   offsets=None if offsets is None else
                                   torch.tensor(offsets, dtype=torch.int32).cuda(), **more)
    assert fg.fft_device_status(None) == fg.FFT_OK
    return grads


def check(fg, args, seed, with_states=True, offsets=None, **more):
    q, k, v, g, beta = args
    batch = q.shape[0] if offsets is None else len(offsets) - 1
    do = normal(seed, *v.shape).to(v.dtype)
    shape = (batch, v.shape[-2], q.shape[-1], v.shape[-1])
    state = 0.3 * normal(seed + 1, *shape) if with_states else None
    dfinal = normal(seed + 2, *shape) if with_states else None
    grads = run(fg, args, do, state, dfinal, offsets, **more)
    for t, like in zip(grads, (q, k, v, g, beta)):
        assert t.dtype == like.dtype and t.shape == like.shape
    want = [[] for _ in NAMES]
    for i in range(batch):
        span = i if offsets is None else slice(offsets[i], offsets[i + 1])
        one = ref.backward(do[span], *(t[span] for t in args), scale=more.get("scale"),
                           state=None if state is None else state[i],
                           dfinal=None if dfinal is None else dfinal[i])
        for w, t in zip(want, one):
            w.append(t)
    for name, got, w in zip(NAMES, grads, want):
        w = torch.stack(w) if offsets is None or name == "dinitial" else torch.cat(w)
        got = got.reshape(w.shape)
        assert got.isfinite().all(), name
        if got.numel():
            tol = HALF_ULP[got.dtype] + (4 * FP if name == "dg" else FP)
            assert rel(got, w) <= tol, (name, rel(got, w), tol)
    return grads


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens", [1, 2, 63, 64, 65, 128, 200])
def test_lengths(fg, kind, tokens):
    check(fg, ref.inputs(1, 2, tokens, 2, 2, 64, 64, TYPES[kind]), 2)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(3, 5), (8, 8), (16, 40), (50, 77), (65, 64), (100, 130), (128, 128), (128, 256),
                                   (96, 300)])
def test_head_sizes(fg, kind, dk, dv):
    check(fg, ref.inputs(3, 1, 150, 1, 2, dk, dv, TYPES[kind]), 4)


@pytest.mark.parametrize("kheads,vheads", [(1, 1), (1, 6), (2, 4), (3, 3)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_shared_key_heads(fg, kind, kheads, vheads):
    check(fg, ref.inputs(5, 2, 100, kheads, vheads, 32, 48, TYPES[kind]), 6)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("offsets", [[0, 64, 128], [0, 1, 1, 65, 66, 200, 200], [0, 0, 0, 5]])
def test_packed(fg, kind, offsets):
    check(fg, [t[0] for t in ref.inputs(7, 1, offsets[-1], 2, 4, 64, 40, TYPES[kind])], 8, offsets=offsets)


def test_without_states_and_with_a_scale(fg):
    check(fg, ref.inputs(9, 2, 90, 1, 1, 32, 32), 10, with_states=False)
    check(fg, ref.inputs(9, 1, 90, 1, 1, 32, 32), 10, scale=-0.7)


def test_extreme_decays_and_strengths(fg):
    q, k, v, g, beta = ref.inputs(11, 1, 300, 2, 2, 64, 64)
    g[0, :100, 0] = 0.0
    g[0, 100:200, 0] = -300.0
    g[0, 150:160, 1] = -500.0
    g[0, 200:, 1] = -1e-6
    beta[0, 50:60] = 0.0            # tokens that write nothing still have a gradient
    beta[0, 60:70] = 1.0
    beta[0, 70:80] = 2.0
    check(fg, (q, k, v, g, beta), 12)


def test_against_differences_of_the_forward_pass(fg):
    # The 64-bit recurrence, central differences along random directions: a step of 1e-4 leaves 1e-8.
    args = [t[0] for t in ref.inputs(13, 1, 70, 1, 2, 8, 12)]
    state, dfinal = 0.3 * normal(1, 2, 8, 12).double(), normal(2, 2, 8, 12)
    do = normal(3, *args[2].shape)
    grads = run(fg, [t[None] for t in args], do[None], state[None].float(), dfinal[None])
    inputs = [t.double() for t in args] + [state.float().double()]

    def value(ts):
        o, s = ref.forward(*ts[:5], state=ts[5])
        return float((o * do).sum() + (s * dfinal).sum())

    for i, grad in enumerate(grads):
        way = normal(20 + i, *inputs[i].shape).double()
        h = 1e-4
        up, down = list(inputs), list(inputs)
        up[i], down[i] = inputs[i] + h * way, inputs[i] - h * way
        slope = (value(up) - value(down)) / (2 * h)
        g64 = grad.double().cpu().reshape(way.shape)
        # 4 FP of the gradient's own size, along a direction of about sqrt(n)
        bound = 4 * FP * float(g64.norm()) * float(way.norm()) / way.numel() ** 0.5 * 4 + 1e-6 * abs(slope) + 1e-6
        assert abs(slope - float((g64 * way).sum())) <= bound, NAMES[i]


def test_rows_beyond_the_sequences_are_not_read_or_written(fg):
    args = [t[0] for t in ref.inputs(14, 1, 200, 1, 2, 64, 64, torch.bfloat16)]
    do = normal(1, *args[2].shape).bfloat16()
    for t in args + [do]:
        t[:10] = float("nan")
        t[150:] = float("nan")
    grads = run(fg, args, do, offsets=[10, 70, 70, 150])
    for i, (a, b) in ((0, (10, 70)), (2, (70, 150))):
        want = ref.backward(do[a:b], *(t[a:b] for t in args))
        for name, got, w in zip(NAMES, grads, want):
            got = got[i] if name == "dinitial" else got[a:b]
            assert rel(got, w) <= HALF_ULP[got.dtype] + (4 * FP if name == "dg" else FP), name


def test_same_bits_again_on_another_stream_and_in_a_graph(fg):
    args = cuda(ref.inputs(15, 2, 300, 2, 4, 128, 128, torch.bfloat16))
    do = normal(1, *args[2].shape).bfloat16().cuda()
    torch.cuda.synchronize()
    runs = []
    for stream in (None, torch.cuda.Stream(), None):
        runs.append(fg.delta_rule_backward(do, *args, stream=stream))
        torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fg.delta_rule_backward(do, *args)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(runs[0], got))


def test_nothing_to_do(fg):
    args = ref.inputs(16, 2, 0, 1, 2, 16, 24)
    dfinal = normal(1, 2, 2, 16, 24)
    grads = run(fg, args, args[2], dfinal=dfinal)
    assert torch.equal(grads[5].cpu(), dfinal) and grads[0].shape == (2, 0, 1, 16)


def test_refusals(fg):
    q, k, v, g, beta = cuda(ref.inputs(17, 1, 5, 2, 4, 16, 16))
    with pytest.raises(ValueError):
        fg.delta_rule_backward(v[:, :4], q, k, v, g, beta)
    with pytest.raises(ValueError):
        fg.delta_rule_backward(v.half(), q, k, v, g, beta)
    with pytest.raises(ValueError):
        fg.delta_rule_backward(v, q, k, v, g, beta, dfinal_state=torch.zeros(1, 4, 16, 15, device="cuda"))
    with pytest.raises(fg.FFTError):
        fg.delta_rule_backward(v[:, :, :3], q, k, v[:, :, :3], g[:, :, :3], beta[:, :, :3])


@pytest.mark.parametrize("kind", list(TYPES))
def test_columns_of_different_size(fg, kind):
    # one scale holds all columns of a head's state: what is small beside the
    # largest is small in every sum over columns too
    q, k, v, g, beta = ref.inputs(31, 1, 200, 1, 2, 64, 96, torch.float32)
    v = v * 2.0 ** -(torch.arange(96) % 13).float()
    check(fg, (q.to(TYPES[kind]), k.to(TYPES[kind]), v.to(TYPES[kind]), g, beta), 32)


@pytest.mark.parametrize("kind,tokens,heads,dv", [("f32", 150, 2, 256), ("f32", 3000, 4, 128), ("bf16", 6000, 4, 128),
                                                  ("bf16", 700, 2, 520)])
def test_same_bits_again(fg, kind, tokens, heads, dv):
    args = cuda(ref.inputs(33, 1, tokens, heads, heads, 128, dv, TYPES[kind]))
    do = normal(34, 1, tokens, heads, dv).to(TYPES[kind]).cuda()
    first = fg.delta_rule_backward(do, *args)
    for _ in range(30):
        for a, b in zip(fg.delta_rule_backward(do, *args), first):
            assert torch.equal(a, b)
    assert fg.fft_device_status(None) == fg.FFT_OK
