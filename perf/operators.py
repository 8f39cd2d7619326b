"""What the sequence-model operators of this library are measured on: the
gated delta rule (whole sequences, their gradients, single tokens), layer
normalisation (forward, backward) and the clipping of gradients by their
global norm.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, with ``own`` set, through the calls
a user makes of the library.  ``exact`` gives the same results in 64 bits
straight from the definitions.
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_CHUNK = 64
_EPS = 1e-5


def listed():
    return [
        # The normalisation in front of one decoding step of a few sequences: latency only.
        dict(name="norm one step", op="norm", rows=4, dim=2048, type="bf16", wtype="bf16"),
        # The same layer over a training batch.
        dict(name="norm batch", op="norm", rows=16384, dim=4096, type="bf16", wtype="f32"),
        # Its gradients, the weight's reduced over all rows.
        dict(name="norm gradient batch", op="norm_grad", rows=16384, dim=4096, type="bf16", wtype="f32"),
        # An odd width in fp32: rows that no vector load fits.
        dict(name="norm gradient odd", op="norm_grad", rows=4099, dim=3001, type="f32", wtype="f32"),
        # One long prompt, value heads grouped over key heads: few heads, a long chain.
        dict(name="delta prompt", op="delta", batch=1, tokens=8192, kheads=16, vheads=32, dk=128, dv=128,
             type="bf16", packed=False, initial=False),
        # Prompts of different lengths (one of them empty, one of a single token) continuing stored states.
        dict(name="delta packed", op="delta", batch=24, tokens=7001, kheads=12, vheads=12, dk=64, dv=64,
             type="f16", packed=True, initial=True),
        # Training step of one layer.
        dict(name="delta gradient", op="delta_grad", batch=4, tokens=16384, kheads=16, vheads=16, dk=128, dv=128,
             type="bf16", packed=False, initial=False),
        # A small packed batch in fp32 with odd head sizes and an initial state that learns.
        dict(name="delta gradient odd", op="delta_grad", batch=5, tokens=1501, kheads=3, vheads=6, dk=50, dv=77,
             type="f32", packed=True, initial=True),
        # One token of one sequence: latency.
        dict(name="delta token", op="step", batch=1, kheads=16, vheads=32, dk=128, dv=128, tokens=1, type="bf16"),
        # One token of each of many sequences, their states scattered in a pool.
        dict(name="delta tokens batch", op="step", batch=128, kheads=16, vheads=32, dk=128, dv=128, tokens=1,
             type="bf16"),
        # Gradients of a small model: many small tensors.
        dict(name="clip small", op="clip", tensors=61, values=400_000, type="f32", max_norm=1.0),
        # Gradients of a large one, matrices and vectors mixed.
        dict(name="clip large", op="clip", tensors=291, values=600_000_000, type="bf16", max_norm=1.0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "delta", "delta_grad", "step", "clip"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "norm_grad"):
        dim = rng.choice([_spread(rng, 64, 16384), 8 * _spread(rng, 16, 1024)])
        rows = _spread(rng, 1, max(2, 30_000_000 // dim))
        return dict(op=op, rows=rows, dim=dim, type=kind, wtype=rng.choice([kind, "f32"]))
    if op == "clip":
        return dict(op=op, tensors=_spread(rng, 1, 400), values=_spread(rng, 1000, 300_000_000), type=kind,
                    max_norm=rng.choice([0.5, 1.0, 1e9]))
    kheads = _spread(rng, 1, 16)
    vheads = kheads * rng.choice([1, 1, 2, 3])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (rng.randint(8, 128), rng.randint(8, 160))])
    if op == "step":
        return dict(op=op, batch=_spread(rng, 1, 100), kheads=kheads, vheads=vheads, dk=dk, dv=dv,
                    tokens=rng.choice([1, 1, 1, 2, 4]), type=kind)
    batch = _spread(rng, 1, 32)
    tokens = _spread(rng, 1, max(2, min(16000, 200_000 // vheads)))
    packed = rng.random() < 0.6
    if not packed:
        tokens = max(1, tokens // batch) * batch
    return dict(op=op, batch=batch, tokens=tokens, kheads=kheads, vheads=vheads, dk=dk, dv=dv, type=kind,
                packed=packed, initial=rng.random() < 0.5)


def _lengths(case):
    """Lengths of a packed batch: uneven, with an empty and a one-token sequence where there is room."""
    batch, total = case["batch"], case["tokens"]
    if not case["packed"]:
        return [total // batch] * batch
    rng = random.Random(batch * 1_000_003 + total)
    cuts = sorted(rng.randint(0, total) for _ in range(batch - 1))
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if batch >= 4 and lengths[0] >= 1:
        lengths[2] += lengths[0] - 1
        lengths[0] = 1
        lengths[3] += lengths[1]
        lengths[1] = 0
    return lengths


def _tensor_sizes(case):
    """Sizes of a model's tensors: half of them vectors, the rest matrices that share what is left."""
    n, left = case["tensors"], case["values"]
    rng = random.Random(n * 1_000_003 + left)
    sizes = []
    for i in range(n - 1):
        part = max(1, left // (n - i))
        size = rng.randint(max(1, part // 200), max(1, part // 50)) if i % 2 else rng.randint(part, part + part // 2 + 1)
        size = max(1, min(size, left - (n - i - 1)))
        sizes.append(size)
        left -= size
    return sizes + [max(1, left)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    op, kind = case["op"], _TYPES[case["type"]]
    state = dict(case=case)
    if op in ("norm", "norm_grad"):
        rows, dim, wkind = case["rows"], case["dim"], _TYPES[case["wtype"]]
        # Activations with a level and a scale of their own in each row.
        x = normal(rows, dim) * (0.5 + normal(rows, 1).abs()) + 0.3 * normal(rows, 1) + 0.2
        state["x"] = x.to(kind)
        state["w"] = (1 + 0.1 * normal(dim)).to(wkind)
        state["b"] = (0.1 * normal(dim)).to(wkind)
        if op == "norm_grad":
            state["dy"] = normal(rows, dim).to(kind)
            x = state["x"].float()
            state["mean"] = x.mean(1)
            state["rstd"] = (x - state["mean"][:, None]).square().mean(1).add(_EPS).rsqrt()
        return state
    if op == "clip":
        sizes = _tensor_sizes(case)
        spread = 3 * math.sqrt(1.0 / case["values"])
        state["grads"] = [(normal(n) * spread * (0.2 + (i % 7))).to(kind) for i, n in enumerate(sizes)]
        state["out"] = [torch.empty_like(t) for t in state["grads"]]
        return state
    batch, kheads, vheads, dk, dv = (case[k] for k in ("batch", "kheads", "vheads", "dk", "dv"))
    total = batch * case["tokens"] if op == "step" else case["tokens"]

    def unit(t):
        return t / t.norm(dim=-1, keepdim=True)

    state["q"] = unit(normal(total, kheads, dk)).to(kind)
    # Keys of one head lean towards a common direction, as learnt ones do.
    state["k"] = unit(normal(total, kheads, dk) + 0.5 * normal(1, kheads, dk)).to(kind)
    state["v"] = normal(total, vheads, dv).to(kind)
    # Log decays from nearly none to a quick forgetting, by head; write strengths between 0 and 1.
    rate = torch.logspace(-2.5, 0.5, vheads, device="cuda")
    state["g"] = -rate * torch.nn.functional.softplus(normal(total, vheads))
    state["beta"] = torch.sigmoid(normal(total, vheads))
    if op == "step":
        pool = batch + batch // 2
        state["pool"] = 0.3 * normal(pool, vheads, dk, dv)
        state["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:batch].int()
        for name in ("q", "k", "v", "g", "beta"):
            state[name] = state[name].reshape(batch, case["tokens"], *state[name].shape[1:])
        return state
    lengths = _lengths(case)
    state["initial"] = 0.3 * normal(batch, vheads, dk, dv) if case["initial"] else None
    if case["packed"]:
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        state["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    else:
        state["offsets"] = None
        for name in ("q", "k", "v", "g", "beta"):
            state[name] = state[name].reshape(batch, lengths[0], *state[name].shape[1:])
    state["longest"] = max(lengths)
    if op == "delta_grad":
        state["do"] = normal(*state["v"].shape).to(kind)
        state["dfinal"] = 0.1 * normal(batch, vheads, dk, dv) if case["initial"] else None
    return state


# ---- the plain forms --------------------------------------------------------------------------------

def _padded(x, state):
    """[batch, whole chunks of tokens, ...] in fp32 of packed or uniform rows, zero where there is no token."""
    batch, longest = state["case"]["batch"], max(1, state["longest"])
    width = -(-longest // _CHUNK) * _CHUNK
    at = torch.arange(width, device=x.device)
    if state["offsets"] is None:
        index, there = at.clamp(max=longest - 1).expand(batch, width), (at < longest).expand(batch, width)
        x = x.float()[torch.arange(batch, device=x.device)[:, None], index]
    else:
        begin, end = state["offsets"][:-1].long(), state["offsets"][1:].long()
        index = begin[:, None] + at
        there = index < end[:, None]
        x = x.float()[torch.where(there, index, 0)]
    return x * there.reshape(batch, width, *([1] * (x.dim() - 2)))


def _unpadded(x, state):
    """The rows of the tokens that there are: the inverse of _padded."""
    if state["offsets"] is None:
        return x[:, : state["longest"]]
    offsets = state["offsets"].long()
    token = torch.arange(state["case"]["tokens"], device=x.device)
    row = torch.searchsorted(offsets[1:].contiguous(), token, right=True)
    return x[row, token - offsets[row]]


def _delta_plain(q, k, v, g, beta, initial, state):
    """Chunks of 64 tokens: inside a chunk by matrix products with the inverse of a unit triangular matrix
    (by doubling its diagonal blocks), from chunk to chunk by the state."""
    case = state["case"]
    batch, heads, dk, dv = case["batch"], case["vheads"], case["dk"], case["dv"]
    group, scale = heads // case["kheads"], case["dk"] ** -0.5
    q, k, v, g, beta = (_padded(t, state) for t in (q, k, v, g, beta))
    q, k = q.repeat_interleave(group, 2), k.repeat_interleave(group, 2)
    # [batch, heads, chunks, 64, ...]
    q, k, v = (t.transpose(1, 2).reshape(batch, heads, -1, _CHUNK, t.shape[-1]) for t in (q, k, v))
    g, beta = (t.transpose(1, 2).reshape(batch, heads, -1, _CHUNK) for t in (g, beta))
    low = torch.ones(_CHUNK, _CHUNK, device=q.device).tril().bool()
    strict = low.tril(-1)
    # Sums of g over (j, i], summed as such: differences of running sums would cancel where g is large.
    between = torch.where(strict, g[..., :, None], 0).cumsum(-2)
    decay = torch.where(low, between, -math.inf).exp()
    total = g.cumsum(-1)
    inner = torch.where(strict, beta[..., :, None] * decay * (k @ k.transpose(-1, -2)), 0)
    size, inverse = 1, torch.eye(_CHUNK, device=q.device)
    while size < _CHUNK:
        at = torch.arange(_CHUNK, device=q.device) // size
        pair = (at[:, None] == at[None, :] + 1) & (at[:, None] % 2 == 1)
        inverse = inverse - inverse @ torch.where(pair, inner, 0) @ inverse
        size *= 2
    mixed = decay * (q @ k.transpose(-1, -2))
    gamma = total.exp()[..., None]
    last = total[..., -1:]
    kd = k * between[..., -1, :].exp()[..., None]
    s = q.new_zeros(batch, heads, dk, dv) if initial is None else initial.float()
    outs = []
    for c in range(q.shape[2]):
        u = inverse[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - gamma[:, :, c] * (k[:, :, c] @ s)))
        outs.append(scale * (gamma[:, :, c] * (q[:, :, c] @ s) + mixed[:, :, c] @ u))
        s = last[:, :, c].exp()[..., None] * s + kd[:, :, c].transpose(-1, -2) @ u
    o = torch.stack(outs, 2).reshape(batch, heads, -1, dv).transpose(1, 2)
    return _unpadded(o, state), s


def _step_plain(state):
    case, pool, slots = state["case"], state["pool"], state["slots"].long()
    group, scale = case["vheads"] // case["kheads"], case["dk"] ** -0.5
    q, k = (state[n].float().repeat_interleave(group, 2) for n in ("q", "k"))
    v, s, outs = state["v"].float(), pool[slots], []
    for t in range(case["tokens"]):
        s = s * state["g"][:, t, :, None, None].exp()
        u = state["beta"][:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * s).sum(2))
        s = s + k[:, t, :, :, None] * u[:, :, None, :]
        outs.append(scale * (q[:, t, :, :, None] * s).sum(2))
    pool[slots] = s
    return {"o": torch.stack(outs, 1).to(state["v"].dtype), "pool": pool}


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "norm":
        x = state["x"].float()
        mean = x.mean(1)
        x = x - mean[:, None]
        rstd = x.square().mean(1).add(_EPS).rsqrt()
        y = x * rstd[:, None] * state["w"].float() + state["b"].float()
        return {"y": y.to(state["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        x, dy, rstd = state["x"].float(), state["dy"].float(), state["rstd"][:, None]
        xh = (x - state["mean"][:, None]) * rstd
        d = dy * state["w"].float()
        dx = rstd * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
        wkind = state["w"].dtype
        return {"dx": dx.to(state["x"].dtype), "dw": (dy * xh).sum(0).to(wkind), "db": dy.sum(0).to(wkind)}
    if op == "clip":
        norm = torch.stack([t.float().square().sum() for t in state["grads"]]).sum().sqrt()
        factor = (case["max_norm"] / (norm + 1e-6)).clamp(max=1)
        return {"norm": norm, "whole": torch.cat([(t.float() * factor).to(t.dtype) for t in state["grads"]])}
    if op == "step":
        return _step_plain(state)
    names = ("q", "k", "v", "g", "beta")
    if op == "delta":
        o, s = _delta_plain(*(state[n] for n in names), state["initial"], state)
        return {"o": o.to(state["v"].dtype), "s": s}
    with torch.enable_grad():
        leaf = {n: state[n].float().requires_grad_() for n in names}
        if state["initial"] is not None:
            leaf["initial"] = state["initial"].detach().requires_grad_()
        o, s = _delta_plain(*(leaf[n] for n in names), leaf.get("initial"), state)
        value = (o * state["do"].float()).sum()
        if state["dfinal"] is not None:
            value = value + (s * state["dfinal"]).sum()
        grads = torch.autograd.grad(value, list(leaf.values()))
    return {"d" + n: d.to(state[n].dtype) for n, d in zip(leaf, grads)}


# ---- the library's ----------------------------------------------------------------------------------

def _run_own(state):
    import fft_convolution_gb300 as fg

    case = state["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = fg.layer_norm(state["x"], state["w"], state["b"], eps=_EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dw, db = fg.layer_norm_backward(state["dy"], state["x"], state["w"], state["mean"], state["rstd"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "clip":
        whole = torch.empty(sum(t.numel() for t in state["grads"]), dtype=state["grads"][0].dtype, device="cuda")
        norm = fg.clip_grad_norm(state["grads"], case["max_norm"],
                                 out=list(whole.split([t.numel() for t in state["grads"]])))
        return {"norm": norm, "whole": whole}
    args = [state[n] for n in ("q", "k", "v", "g", "beta")]
    if op == "step":
        o = fg.delta_rule_step(*args, state["pool"], slots=state["slots"])
        return {"o": o, "pool": state["pool"]}
    if op == "delta":
        o, s = fg.delta_rule(*args, initial_state=state["initial"], offsets=state["offsets"])
        return {"o": o, "s": s}
    grads = fg.delta_rule_backward(state["do"], *args, initial_state=state["initial"], offsets=state["offsets"],
                                   dfinal_state=state["dfinal"])
    names = ("dq", "dk", "dv", "dg", "dbeta", "dinitial")
    return {n: d for n, d in zip(names, grads) if n != "dinitial" or state["initial"] is not None}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- work -------------------------------------------------------------------------------------------

def work(case):
    size = 4 if case["type"] == "f32" else 2
    op = case["op"]
    if op in ("norm", "norm_grad"):
        wsize, n = 4 if case["wtype"] == "f32" else 2, case["rows"] * case["dim"]
        if op == "norm":
            return dict(bytes=2 * n * size + 2 * case["dim"] * wsize + 8 * case["rows"], flops=8 * n)
        return dict(bytes=3 * n * size + 3 * case["dim"] * wsize + 8 * case["rows"], flops=14 * n)
    if op == "clip":
        return dict(bytes=2 * size * case["values"], flops=3 * case["values"])
    total = case["tokens"] * (case["batch"] if op == "step" else 1)
    kv = case["dk"] * case["dv"]
    qk = total * case["kheads"] * case["dk"] * size * 2
    v = total * case["vheads"] * case["dv"] * size
    gates = total * case["vheads"] * 8
    states = case["batch"] * case["vheads"] * kv * 4
    if op == "step":  # each state once in, once out
        return dict(bytes=qk + 2 * v + gates + 2 * states, flops=7 * total * case["vheads"] * kv)
    if op == "delta":
        return dict(bytes=qk + 2 * v + gates + states * (2 if case["initial"] else 1),
                    flops=6 * total * case["vheads"] * kv)
    return dict(bytes=2 * qk + 3 * v + 2 * gates + (3 * states if case["initial"] else 0),
                flops=16 * total * case["vheads"] * kv)


# ---- from the definitions, in 64 bits ------------------------------------------------------------------

def _exact_delta(q, k, v, g, beta, s, scale, do=None, dfinal=None):
    """One token after the other over [time, batch, heads, ...]; with `do` the gradients too, by the same recurrence
    run backwards over the states that the forward run left."""
    keep, outs = [], []
    for t in range(q.shape[0]):
        keep.append(s)
        s = s * g[t].exp()[..., None, None]
        u = beta[t][..., None] * (v[t] - torch.einsum("bhkv,bhk->bhv", s, k[t]))
        s = s + k[t][..., :, None] * u[..., None, :]
        if do is None:
            keep.clear()
            outs.append(scale * torch.einsum("bhkv,bhk->bhv", s, q[t]))
    if do is None:
        return (torch.stack(outs) if outs else torch.zeros_like(v)), s
    d = torch.zeros_like(s) if dfinal is None else dfinal
    grads = [torch.zeros_like(t) for t in (q, k, v, g, beta)]
    for t in reversed(range(q.shape[0])):
        alpha = g[t].exp()[..., None, None]
        before = keep[t] * alpha
        miss = v[t] - torch.einsum("bhkv,bhk->bhv", before, k[t])
        u = beta[t][..., None] * miss
        after = before + k[t][..., :, None] * u[..., None, :]
        grads[0][t] = scale * torch.einsum("bhkv,bhv->bhk", after, do[t])
        d = d + scale * q[t][..., :, None] * do[t][..., None, :]
        du = torch.einsum("bhkv,bhk->bhv", d, k[t])
        dy = beta[t][..., None] * du
        grads[1][t] = torch.einsum("bhkv,bhv->bhk", d, u) - torch.einsum("bhkv,bhv->bhk", before, dy)
        grads[2][t] = dy
        grads[4][t] = (du * miss).sum(-1)
        d = d - k[t][..., :, None] * dy[..., None, :]
        grads[3][t] = (d * before).sum((-1, -2))
        d = d * alpha
        keep[t] = None
    return grads, d


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        x, w, b = (state[n].double() for n in ("x", "w", "b"))
        mean = x.mean(1, keepdim=True)
        var = ((x - mean) ** 2).mean(1, keepdim=True)
        if op == "norm":
            rstd = 1 / torch.sqrt(var + _EPS)
            return {"y": (x - mean) * rstd * w + b, "mean": mean[:, 0], "rstd": rstd[:, 0]}
        mean, rstd, dy = state["mean"].double()[:, None], state["rstd"].double()[:, None], state["dy"].double()
        n = x.shape[1]
        normed, pulled = (x - mean) * rstd, dy * w
        along = (pulled * normed).sum(1, keepdim=True) / n
        dx = (pulled - pulled.sum(1, keepdim=True) / n - normed * along) * rstd
        return {"dx": dx, "dw": torch.einsum("rd,rd->d", dy, normed), "db": dy.sum(0)}
    if op == "clip":
        whole = torch.cat([t.double() for t in state["grads"]])
        norm = (whole ** 2).sum() ** 0.5
        return {"norm": norm, "whole": whole * min(1.0, case["max_norm"] / (float(norm) + 1e-6))}
    group, scale = case["vheads"] // case["kheads"], 1 / math.sqrt(case["dk"])
    names = ["q", "k", "v", "g", "beta"]
    if op == "step":
        args = [state[n].double().transpose(0, 1) for n in names]
        args[:2] = [t.repeat_interleave(group, 2) for t in args[:2]]
        pool, slots = state["pool"].double(), state["slots"].long()
        o, s = _exact_delta(*args, pool[slots], scale)
        pool[slots] = s
        return {"o": o.transpose(0, 1), "pool": pool}
    batch, heads, dk, dv = case["batch"], case["vheads"], case["dk"], case["dv"]
    lengths = _lengths(case)
    # All sequences advance together: time first, a sequence that has ended stands still (no write, no decay).
    if max(lengths) * batch * heads * dk * dv * 8 > 150e9 and op == "delta_grad":
        return None
    steps, flat, begin = max(lengths), {}, 0
    if op == "delta_grad":
        names.append("do")
    for n in names:
        t = state[n].double().reshape(case["tokens"], *state[n].shape[-(1 if n in ("g", "beta") else 2):])
        flat[n] = t.new_zeros(steps, batch, *t.shape[1:])
    for i, length in enumerate(lengths):
        for n in names:
            t = state[n].reshape(case["tokens"], *flat[n].shape[2:])
            flat[n][:length, i] = t[begin: begin + length].double()
        begin += length
    for n in ("q", "k"):
        flat[n] = flat[n].repeat_interleave(group, 2)
    s = torch.zeros(batch, heads, dk, dv, dtype=torch.float64, device="cuda")
    if state["initial"] is not None:
        s = state["initial"].double()

    def rows(t, like):
        return torch.cat([t[:length, i] for i, length in enumerate(lengths)]).reshape(like.shape)

    args = [flat[n] for n in ("q", "k", "v", "g", "beta")]
    if op == "delta":
        o, s = _exact_delta(*args, s, scale)
        return {"o": rows(o, state["v"]), "s": s}
    dfinal = None if state["dfinal"] is None else state["dfinal"].double()
    grads, ds = _exact_delta(*args, s, scale, flat["do"], dfinal)
    for i in (0, 1):  # heads that share a key head share its gradient
        t = grads[i]
        grads[i] = t.reshape(*t.shape[:2], -1, group, dk).sum(3)
    found = {"d" + n: rows(t, state[n]) for n, t in zip(names, grads)}
    if state["initial"] is not None:
        found["dinitial"] = ds
    return found
