"""GPU gated delta rule (whole sequences and single tokens) against the
token-by-token recurrence in 64 bits.

Tolerances (relative L2), fixed before the first run: every factor of a
product that is not exactly bf16 keeps 16 significand bits or more (2^-18 of
rounding on average over signs), and an output passes through at most five
products one after the other: FP = 5 * 2^-18 = 1.9e-5 for what is returned
in fp32.  An output rounded to p bits adds 2^-p.  Single tokens are computed
in fp32 throughout: 64 * 2^-24.
"""
import pytest

torch = pytest.importorskip("torch")
import delta_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FP = 5 * 2.0 ** -18


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


def state_like(seed, batch, vheads, dk, dv):
    return 0.3 * torch.randn(batch, vheads, dk, dv, generator=torch.Generator().manual_seed(seed))


def check(fg, args, state=None, offsets=None, fp=FP, **more):
    """delta_rule on CPU inputs against the recurrence, sequence by sequence."""
    o, s = fg.delta_rule(*cuda(args), initial_state=None if state is None else state.cuda(),
                         offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda(),
                         **more)
    assert fg.fft_device_status(None) == fg.FFT_OK
    kind = args[2].dtype
    assert o.dtype == kind and o.shape == args[2].shape and s.dtype == torch.float32
    spans = [(i, slice(None)) for i in range(args[0].shape[0])] if offsets is None else \
        [(i, slice(a, b)) for i, (a, b) in enumerate(zip(offsets, offsets[1:]))]
    for i, span in spans:
        one = [t[i] if offsets is None else t[span] for t in args]
        o64, s64 = ref.forward(*one, scale=more.get("scale"), state=None if state is None else state[i])
        got = o[i] if offsets is None else o[span]
        assert got.isfinite().all() and s[i].isfinite().all()
        if got.numel():
            assert rel(got, o64) <= HALF_ULP[kind] + fp, (i, rel(got, o64))
        assert rel(s[i], s64) <= fp, (i, rel(s[i], s64))
    return o, s


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens", [1, 2, 63, 64, 65, 128, 200, 321])
def test_lengths(fg, kind, tokens):
    check(fg, ref.inputs(1, 2, tokens, 2, 2, 64, 64, TYPES[kind]))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (8, 8), (16, 40), (50, 77), (64, 64), (65, 64), (100, 130),
                                   (128, 128), (128, 256), (96, 300)])
def test_head_sizes(fg, kind, dk, dv):
    check(fg, ref.inputs(2, 1, 150, 1, 2, dk, dv, TYPES[kind]), state_like(3, 1, 2, dk, dv))


@pytest.mark.parametrize("kheads,vheads", [(1, 1), (1, 6), (2, 4), (3, 3), (4, 12)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_head_groups(fg, kind, kheads, vheads):
    check(fg, ref.inputs(4, 2, 100, kheads, vheads, 32, 48, TYPES[kind]), state_like(5, 2, vheads, 32, 48))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("offsets", [[0, 64, 128], [0, 1, 1, 65, 66, 200, 200], [0, 0, 0, 5], [0, 300],
                                     [0, 63, 127, 191, 255, 256]])
def test_packed(fg, kind, offsets):
    args = [t[0] for t in ref.inputs(6, 1, offsets[-1], 2, 4, 64, 40, TYPES[kind])]
    check(fg, args, state_like(7, len(offsets) - 1, 4, 64, 40), offsets)


def test_many_packed_sequences(fg):
    # more sequences than the threads that lay out the chunks
    lengths = [(i * 7) % 5 for i in range(2500)]
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    args = [t[0] for t in ref.inputs(8, 1, offsets[-1], 1, 1, 8, 8)]
    state = state_like(9, len(lengths), 1, 8, 8)
    o, s = fg.delta_rule(*cuda(args), initial_state=state.cuda(),
                         offsets=torch.tensor(offsets, dtype=torch.int64).cuda())
    for i in list(range(0, 2500, 83)) + [1023, 1024, 1025, 2499]:
        a, b = offsets[i], offsets[i + 1]
        o64, s64 = ref.forward(*(t[a:b] for t in args), state=state[i])
        assert rel(s[i], s64) <= FP
        if b > a:
            assert rel(o[a:b], o64) <= FP


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_same_as_uniform(fg, kind):
    args = ref.inputs(10, 3, 130, 2, 2, 128, 64, TYPES[kind])
    o, s = fg.delta_rule(*cuda(args))
    flat = [t.reshape(390, *t.shape[2:]).cuda() for t in args]
    o2, s2 = fg.delta_rule(*flat, offsets=torch.tensor([0, 130, 260, 390], dtype=torch.int32).cuda())
    assert torch.equal(o.reshape(o2.shape), o2) and torch.equal(s, s2)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strides(fg, kind):
    # q, k, v as slices of one projection (unaligned for the odd size), and as [batch, heads, tokens, *]
    for dk, dv in ((64, 64), (24, 40), (33, 20)):
        q, k, v, g, beta = ref.inputs(11, 2, 100, 2, 2, dk, dv, TYPES[kind])
        whole = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], -1).cuda()
        qs = whole[..., : 2 * dk].unflatten(-1, (2, dk))
        ks = whole[..., 2 * dk: 4 * dk].unflatten(-1, (2, dk))
        vs = whole[..., 4 * dk:].unflatten(-1, (2, dv))
        want = fg.delta_rule(*cuda([q, k, v, g, beta]))
        got = fg.delta_rule(qs, ks, vs, g.cuda(), beta.cuda())
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        t = [x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v, g, beta)]
        assert all(torch.equal(a, b) for a, b in zip(want, fg.delta_rule(*t)))


def test_extreme_decays_and_strengths(fg):
    q, k, v, g, beta = ref.inputs(12, 1, 300, 2, 2, 64, 64)
    g[0, :100, 0] = 0.0
    g[0, 100:200, 0] = -1e30
    g[0, 70, 1] = -float("inf")     # drops the state
    g[0, 150:160, 1] = -500.0
    g[0, 200:, 1] = -1e-6
    beta[0, 50:60] = 0.0            # tokens that write nothing
    beta[0, 60:70] = 1.0
    beta[0, 70:80] = 2.0            # reflections
    check(fg, (q, k, v, g, beta), state_like(1, 1, 2, 64, 64))


def test_repeated_keys(fg):
    # One key throughout: the matrix to invert is full below its diagonal.  Its inverse's entries stay
    # bounded by 1 here (beta <= 1), a power series of it would not.
    q, k, v, g, beta = ref.inputs(13, 1, 200, 1, 1, 64, 64)
    k = k[:, :1].expand_as(k).contiguous()
    check(fg, (q, k, v, torch.zeros_like(g), torch.ones_like(beta)))
    check(fg, (q, k, v, 0.01 * g, beta))


def test_a_fast_head_keeps_its_digits(fg):
    # running sums of g near -1000 within a chunk: their differences must not be taken in fp32
    q, k, v, g, beta = ref.inputs(14, 1, 256, 1, 1, 64, 64)
    g = torch.full_like(g, -20.0)
    g[0, ::2] = -0.01
    check(fg, (q, k, v, g, beta))


def test_scale_and_no_decay(fg):
    args = ref.inputs(15, 1, 90, 1, 1, 32, 32)
    check(fg, args, scale=1.0)
    check(fg, args, scale=-0.25)


def test_rows_beyond_the_sequences_are_not_read(fg):
    args = [t[0] for t in ref.inputs(16, 1, 200, 1, 2, 64, 64, torch.bfloat16)]
    bad = [t.clone() for t in args]
    for t in bad:
        t[:10] = float("nan")
        t[70:80] = float("inf")
        t[150:] = float("nan")
    # sequences 10 .. 70 and 80 .. 150 by offsets whose ends the neighbours' rows touch
    for t in bad:
        t[70:80] = 0
    offsets = torch.tensor([10, 70, 80, 150], dtype=torch.int32).cuda()
    out = torch.full((200, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    o, s = fg.delta_rule(*cuda(bad), offsets=offsets, out=out)
    for i, (a, b) in ((0, (10, 70)), (2, (80, 150))):
        o64, s64 = ref.forward(*(t[a:b] for t in bad))
        assert rel(o[a:b], o64) <= HALF_ULP[torch.bfloat16] + FP and rel(s[i], s64) <= FP
    assert (o[:10] == 5).all() and (o[150:] == 5).all()


def test_a_value_that_is_not_finite_stays_in_its_sequence_and_head(fg):
    args = ref.inputs(17, 2, 200, 2, 2, 64, 64)
    args[2][0, 70, 1, 3] = float("nan")
    o, s = fg.delta_rule(*cuda(args))
    clean = ref.inputs(17, 2, 200, 2, 2, 64, 64)
    o2, s2 = fg.delta_rule(*cuda(clean))
    assert torch.equal(o[1], o2[1]) and torch.equal(o[0, :, 0], o2[0, :, 0])
    assert torch.equal(o[0, :64, 1], o2[0, :64, 1]) and torch.isnan(s[0, 1]).any()
    assert torch.equal(s[1], s2[1]) and torch.equal(s[0, 0], s2[0, 0])


def test_offsets_out_of_order_stay_in_bounds(fg):
    args = [t[0].cuda() for t in ref.inputs(18, 1, 100, 1, 1, 16, 16)]
    for offsets in ([0, 500, 20, 100], [-5, 10, 1 << 30], [90, 10, 50]):
        o, s = fg.delta_rule(*args, offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert fg.fft_device_status(None) == fg.FFT_OK and s.isfinite().all()


def test_nothing_to_do(fg):
    args = cuda(ref.inputs(19, 2, 0, 1, 2, 16, 24))
    state = state_like(1, 2, 2, 16, 24).cuda()
    o, s = fg.delta_rule(*args, initial_state=state)
    assert o.shape == (2, 0, 2, 24) and torch.equal(s, state)
    o, s = fg.delta_rule(*args)
    assert not s.any()
    o, s = fg.delta_rule(*cuda(ref.inputs(19, 0, 5, 1, 2, 16, 24)))
    assert o.numel() == 0 and s.shape == (0, 2, 16, 24)


def test_state_carries_over(fg):
    args = cuda(ref.inputs(20, 2, 300, 2, 4, 64, 64))
    o, s = fg.delta_rule(*args)
    o1, s1 = fg.delta_rule(*(t[:, :137] for t in args))
    o2, s2 = fg.delta_rule(*(t[:, 137:] for t in args), initial_state=s1)
    assert rel(torch.cat([o1, o2], 1), o) <= 2 * FP and rel(s2, s) <= 2 * FP


def test_same_bits_again_on_another_stream_and_in_a_graph(fg):
    args = cuda(ref.inputs(21, 2, 300, 2, 4, 128, 128, torch.bfloat16))
    torch.cuda.synchronize()
    runs = []
    for stream in (None, torch.cuda.Stream(), None):
        runs.append(fg.delta_rule(*args, stream=stream))
        torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
    graph = torch.cuda.CUDAGraph()
    offsets = torch.tensor([0, 100, 600], dtype=torch.int32).cuda()
    flat = [t.flatten(0, 1) for t in args]
    want = fg.delta_rule(*flat, offsets=offsets)
    with torch.cuda.graph(graph):
        got = fg.delta_rule(*flat, offsets=offsets)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# ---- single tokens -------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("tokens", [1, 2, 5])
@pytest.mark.parametrize("kheads,vheads,dk,dv", [(1, 1, 1, 1), (2, 4, 64, 64), (1, 3, 50, 77), (2, 2, 128, 128),
                                                 (1, 2, 200, 33), (1, 1, 256, 130)])
def test_step(fg, kind, tokens, kheads, vheads, dk, dv):
    args = ref.inputs(30, 3, tokens, kheads, vheads, dk, dv, TYPES[kind])
    state = state_like(31, 3, vheads, dk, dv)
    pool = state.cuda()
    o = fg.delta_rule_step(*cuda(args), pool)
    for i in range(3):
        o64, s64 = ref.forward(*(t[i] for t in args), state=state[i])
        assert rel(o[i], o64) <= HALF_ULP[TYPES[kind]] + 64 * 2.0 ** -24
        assert rel(pool[i], s64) <= 64 * 2.0 ** -24


def test_step_slots(fg):
    args = ref.inputs(32, 4, 1, 1, 2, 64, 64)
    state = state_like(33, 6, 2, 64, 64)
    pool = state.cuda()
    slots = [5, -1, 0, 9]  # two idle sequences
    o = fg.delta_rule_step(*cuda(args), pool, slots=torch.tensor(slots, dtype=torch.int32).cuda())
    assert not o[1].any() and not o[3].any()
    for i, slot in ((0, 5), (2, 0)):
        o64, s64 = ref.forward(*(t[i] for t in args), state=state[slot])
        assert rel(o[i], o64) <= 64 * 2.0 ** -24 and rel(pool[slot], s64) <= 64 * 2.0 ** -24
    for slot in (1, 2, 3, 4):
        assert torch.equal(pool[slot].cpu(), state[slot])


def test_step_follows_a_prompt(fg):
    args = cuda(ref.inputs(34, 2, 140, 2, 2, 64, 128))
    o, s = fg.delta_rule(*args)
    o1, pool = fg.delta_rule(*(t[:, :137] for t in args))
    outs = [fg.delta_rule_step(*(t[:, i:i + 1] for t in args), pool) for i in range(137, 140)]
    assert rel(torch.cat(outs, 1), o[:, 137:]) <= 2 * FP and rel(pool, s) <= 2 * FP


def test_step_drops_the_state_and_strides(fg):
    q, k, v, g, beta = ref.inputs(35, 2, 1, 1, 2, 64, 64)
    g[0] = -float("inf")
    state = state_like(36, 2, 2, 64, 64)
    pool = state.cuda()
    t = [x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v, g, beta)]
    o = fg.delta_rule_step(*t, pool)
    for i in range(2):
        o64, s64 = ref.forward(q[i], k[i], v[i], g[i], beta[i], state=state[i])
        assert rel(o[i], o64) <= 64 * 2.0 ** -24 and rel(pool[i], s64) <= 64 * 2.0 ** -24


def test_refusals(fg):
    q, k, v, g, beta = cuda(ref.inputs(40, 1, 5, 2, 4, 16, 16))
    with pytest.raises(ValueError):
        fg.delta_rule(q, k[:, :, :1], v, g, beta)
    with pytest.raises(ValueError):
        fg.delta_rule(q, k, v, g[:, :4], beta)
    with pytest.raises(TypeError):
        fg.delta_rule(q, k, v.half(), g, beta)
    with pytest.raises(TypeError):
        fg.delta_rule(q, k, v, g.double(), beta)
    with pytest.raises(ValueError):
        fg.delta_rule(q, k, v, g, beta.cpu())
    with pytest.raises(ValueError):
        fg.delta_rule(q, k, v, g, beta, initial_state=torch.zeros(1, 4, 16, 15, device="cuda"))
    with pytest.raises(fg.FFTError):  # 3 value heads over 2 key heads
        fg.delta_rule(q, k, v[:, :, :3], g[:, :, :3], beta[:, :, :3])
    with pytest.raises(fg.FFTError):
        fg.delta_rule(q.double(), k.double(), v.double(), g, beta)
    with pytest.raises(fg.FFTError):
        fg.delta_rule(q, k, v, g, beta, scale=float("nan"))
    wide = torch.zeros(1, 5, 2, 129, device="cuda")
    with pytest.raises(fg.FFTError):
        fg.delta_rule(wide, wide, v, g, beta)
    pool = torch.zeros(1, 4, 16, 16, device="cuda")
    with pytest.raises(ValueError):
        fg.delta_rule_step(q, k, v, g, beta, pool.transpose(2, 3))
    with pytest.raises(ValueError):
        fg.delta_rule_step(q, k, v, g, beta, pool, slots=torch.zeros(1, dtype=torch.int64, device="cuda"))
    two = cuda(ref.inputs(40, 2, 1, 2, 4, 16, 16))
    with pytest.raises(fg.FFTError):  # two sequences, one state
        fg.delta_rule_step(*two, pool)
