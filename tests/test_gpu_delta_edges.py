"""The gated delta rule where operands differ much in size, against the
token-by-token recurrence in 64 bits.
"""
import pytest

torch = pytest.importorskip("torch")
import delta_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


# ---- what an output keeps of a sum whose terms are larger than it ------------------------
#
# Every factor of a product keeps 22 significand bits or is exact (2^-23 of rounding), and the tensor
# cores cut each of up to 24 partial sums below the last fp32 bit (2^-23): 32 * 2^-23 of the sum of
# the terms' absolute values, on each output, beside the output's own rounding.
KEPT = 32 * 2.0 ** -23


def outputs_and_terms(q, k, v, g, beta, state):
    """o of one sequence [tokens, heads, dv] in 64 bits, and for each value the sum of the absolute
    values that make it up: |S0|^T |q| as it decays, and |u_j| |k_j . q_t| of the tokens since."""
    q, k, v, g, beta, s = (t.double() for t in (q, k, v, g, beta, state))
    group = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    scale = q.shape[-1] ** -0.5
    first, decay, us, outs, sizes = s.abs(), torch.zeros_like(g[0]), [], [], []
    for t in range(q.shape[0]):
        s = s * g[t].exp()[:, None, None]
        u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", s, k[t]))
        s = s + k[t][:, :, None] * u[:, None, :]
        decay = decay + g[t]
        us.append((u, k[t], decay))
        outs.append(scale * torch.einsum("hkv,hk->hv", s, q[t]))
        size = decay.exp()[:, None] * torch.einsum("hkv,hk->hv", first, q[t].abs())
        for uj, kj, dj in us:
            size = size + ((decay - dj).exp() * (kj * q[t]).sum(-1).abs())[:, None] * uj.abs()
        sizes.append(scale * size)
    return torch.stack(outs), torch.stack(sizes)


def check_terms(fg, args, state):
    o, _ = fg.delta_rule(*cuda([t[None] for t in args]), initial_state=state[None].cuda())
    want, size = outputs_and_terms(*args, state)
    bound = HALF_ULP[o.dtype] * want.abs() + KEPT * size
    off = ((o[0].double().cpu() - want).abs() / bound).max()
    assert off <= 1, float(off)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("dk", [64, 128])
def test_a_small_value_overwrites_a_large_one(fg, kind, dk):
    # q = k, beta = 1: o = scale v (if |k| = 1), where S0^T k is a thousand times as large
    q, k, v, g, beta = (t[0] for t in ref.inputs(51, 1, 100, 1, 1, dk, 64, TYPES[kind]))
    state = 1024 * normal(52, 1, dk, 64)
    check_terms(fg, (k, k, v, torch.zeros_like(g), torch.ones_like(beta)), state)


@pytest.mark.parametrize("kind", list(TYPES))
def test_one_value_among_larger_ones(fg, kind):
    # 64 orthonormal keys (Hadamard's, exact in every type); of the values stored under them one is
    # a thousand times smaller, and that one is read
    h = torch.ones(1, 1)
    while h.shape[0] < 64:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    keys, values = h / 8, 1000 * normal(53, 64, 64)
    values[5] /= 1000
    state = torch.einsum("jk,jv->kv", keys, values)[None]
    q = keys[5].expand(100, 1, 64).to(TYPES[kind]).contiguous()
    _, k, v, g, beta = (t[0] for t in ref.inputs(54, 1, 100, 1, 1, 64, 64, TYPES[kind]))
    k = torch.where(torch.arange(64) < 32, k, torch.zeros_like(k))
    check_terms(fg, (q, k, v, 0.01 * g, 0.1 * beta), state)


# ---- one token after a strong decay ----------------------------------------------------------

# The new state is e^g S + k u in fp32, u = beta (v - e^g S^T k): a sum over dk, rounded a few
# times (64 * 2^-24, as for any single token), at the size of the two terms of each result.
TOKEN = 64 * 2.0 ** -24


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1.0, 1000.0])
@pytest.mark.parametrize("strength", [0.0, 0.01, 0.5])
@pytest.mark.parametrize("dk,dv", [(128, 128), (50, 77), (200, 64)])
def test_step_after_a_strong_decay(fg, kind, size, strength, dk, dv):
    decays = torch.tensor([0.0, -0.1, -0.69, -0.7, -1.0, -5.0, -10.0, -16.0, -60.0, -float("inf")])
    heads = len(decays)
    q, k, v, g, beta = ref.inputs(61, 2, 1, heads, heads, dk, dv, TYPES[kind])
    g, beta = decays.expand(2, 1, heads).contiguous(), torch.full_like(beta, strength)
    state = size * normal(62, 2, heads, dk, dv)
    pool = state.cuda()
    o = fg.delta_rule_step(*cuda((q, k, v, g, beta)), pool)
    scale = dk ** -0.5
    for i in range(2):
        o64, s64 = ref.forward(*(t[i] for t in (q, k, v, g, beta)), state=state[i])
        for h in range(heads):
            e, kh, qh = float(decays[h].double().exp()), k[i, 0, h].double(), q[i, 0, h].double()
            held = e * state[i, h].double()
            u = strength * (v[i, 0, h].double() - held.t() @ kh)
            # S: the errors of u enter along k, those of e^g S stay where they are
            size_u = strength * (v[i, 0, h].double().norm() + (held.t() @ kh).norm())
            bound = TOKEN * (held.norm() + size_u * kh.norm())
            assert float((pool[i, h].double().cpu() - s64[h]).norm()) <= float(bound), (i, h)
            bound = HALF_ULP[TYPES[kind]] * o64[0, h].norm() + TOKEN * scale * (
                (held.t() @ qh).norm() + (kh @ qh).abs() * size_u)
            assert float((o[i, 0, h].double().cpu() - o64[0, h]).norm()) <= float(bound), (i, h)
            assert u.isfinite().all()


# ---- chunks that write nothing, and sizes far apart -----------------------------------------

FP = 5 * 2.0 ** -18          # whole sequences, forward: five products one after the other
FP_GRAD = 12 * 2.0 ** -20    # gradients: twelve
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinitial")


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def check_by_chunk(fg, args, state):
    """Outputs chunk by chunk and the final state, of one sequence."""
    o, s = fg.delta_rule(*cuda(args), initial_state=state.cuda())
    o64, s64 = ref.forward(*(t[0] for t in args), state=state[0])
    for c in range(0, o.shape[1], 64):
        got = o[0, c:c + 64]
        assert got.isfinite().all(), c
        assert rel(got, o64[c:c + 64]) <= HALF_ULP[o.dtype] + FP, c
    assert s.isfinite().all() and rel(s[0], s64) <= FP


def check_gradients(fg, args, do, state, dfinal):
    grads = fg.delta_rule_backward(do.cuda(), *cuda(args), initial_state=state.cuda(),
                                   dfinal_state=None if dfinal is None else dfinal.cuda())
    want = ref.backward(do[0], *(t[0] for t in args), state=state[0], dfinal=None if dfinal is None else dfinal[0])
    for name, got, w in zip(NAMES, grads, want):
        assert got.isfinite().all(), name
        tol = HALF_ULP[got.dtype] + (4 if name == "dg" else 1) * FP_GRAD
        assert rel(got[0], w) <= tol, (name, rel(got[0], w))


def still_chunk(kind, how):
    """Three chunks, the second of them without a write."""
    q, k, v, g, beta = ref.inputs(71, 1, 192, 1, 1, 64, 64, torch.float32)
    beta[:, 64:128] = 0.0
    if how == "small keys":
        k[:, 64:128] *= 2.0 ** (-20 if kind == "f16" else -30)
    elif how == "orthogonal":  # but for a rounding
        q[:, 64:128, :, 32:] = 0.0
        k[:, 64:128, :, :32] = 0.0
        k[:, 64:128, :, 0] = 2.0 ** -24
    return [t.to(TYPES[kind]) for t in (q, k, v)] + [0.01 * g, beta]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("how", ["small keys", "orthogonal", "plain"])
def test_a_chunk_that_writes_nothing(fg, kind, how):
    args = still_chunk(kind, how)
    state = 2.0 ** (11 if kind == "f16" else 14) * normal(72, 1, 1, 64, 64)  # (gradients within fp16's range)
    check_by_chunk(fg, args, state)
    check_gradients(fg, args, normal(73, *args[2].shape).to(TYPES[kind]), state, normal(74, 1, 1, 64, 64))


@pytest.mark.parametrize("how", ["small keys", "orthogonal", "plain", "dropped"])
def test_a_chunk_that_writes_nothing_to_a_very_large_state(fg, how):
    # what the outputs and the states are scaled by lies far apart
    args = still_chunk("f32", how)
    if how == "dropped":  # and nothing to store either
        args[2][:, 64:128] = 0.0
        args[3][:, 64] = -float("inf")
    check_by_chunk(fg, args, 2.0 ** 45 * normal(75, 1, 1, 64, 64))


@pytest.mark.parametrize("how", ["no keys", "no queries", "no gradient", "large queries"])
def test_gradients_of_sizes_far_apart(fg, how):
    args = still_chunk("f32", "plain")
    do, state, dfinal = normal(76, 1, 192, 1, 64), normal(77, 1, 1, 64, 64), None
    if how == "no keys":
        args[1][:, 64:] = 0.0
        do *= 2.0 ** 45
    elif how == "no queries":
        args[0][:, 64:] = 0.0
        do *= 2.0 ** 45
    elif how == "no gradient":
        do[:, 64:] = 0.0
        args[0][:, 64:] *= 2.0 ** 40
        dfinal = normal(78, 1, 1, 64, 64)
    else:
        args[0][:] *= 2.0 ** 40
        args[4][:] = 0.0
    check_gradients(fg, args, do, state, dfinal)


# One scale per column of v holds a chunk, from a bound on what its tokens see: 2^7 to 2^8 times the
# largest value of the state here (2 DK, keys of 1/4).  Scaled to 2^14, fp16 pairs end at 2^-25: 2^-31
# of that value for each of the operands that one after the other carry a result of size 1 (Y, U, W),
# whose rounding adds up over the row sums of the inverse (below 3): 2^-28.
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("larger", [0, 8, 12, 16])
def test_what_a_dropped_state_leaves_in_its_chunk(fg, kind, larger):
    q, k, v, g, beta = ref.inputs(81, 1, 100, 1, 2, 64, 64, TYPES[kind])
    g[0, 32, :] = -float("inf")
    state = 2.0 ** larger * normal(82, 1, 2, 64, 64)
    o, s = fg.delta_rule(*cuda((q, k, v, g, beta)), initial_state=state.cuda())
    o64, s64 = ref.forward(*(t[0] for t in (q, k, v, g, beta)), state=state[0])
    bound = FP + 2.0 ** (larger - 28)
    assert rel(s[0], s64) <= bound
    for part in (slice(0, 32), slice(32, 64), slice(64, 100)):
        assert rel(o[0, part], o64[part]) <= HALF_ULP[o.dtype] + bound, part
