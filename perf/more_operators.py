"""What the operators around a recurrent language model's mixers are measured
on: the embedding of tokens with its gradient, the gated linear recurrence
(whole sequences, its gradients, single tokens), and the cross entropy of a
linear layer over the vocabulary with its gradients.

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


def listed():
    return [
        # Tokens of a training batch into activations.
        dict(name="embed batch", op="embed", tokens=16384, vocabulary=65536, dim=2048, type="bf16", padded=False),
        # The table's gradient in the same step: frequent tokens hundreds of times, most of the table never.
        dict(name="embed gradient batch", op="embed_grad", tokens=16384, vocabulary=65536, dim=2048, type="bf16",
             padded=False, added=False),
        # A ragged batch in fp32 with padding, added to the gradient that a tied output layer has left.
        dict(name="embed gradient added odd", op="embed_grad", tokens=5003, vocabulary=30011, dim=1001, type="f32",
             padded=True, added=True),
        # One long prompt: few lanes, a long axis.
        dict(name="scan prompt", op="scan", batch=1, tokens=32768, channels=4096, type="bf16", gtype="bf16",
             gated=True, packed=False, initial=False),
        # Prompts of different lengths (one of them empty, one of a single token) continuing stored states.
        dict(name="scan packed", op="scan", batch=24, tokens=7001, channels=1280, type="f16", gtype="f32",
             gated=True, packed=True, initial=True),
        # Training step of one layer.
        dict(name="scan gradient", op="scan_grad", batch=8, tokens=32768, channels=2048, type="bf16", gtype="bf16",
             gated=True, packed=False, initial=False),
        # A small packed batch in fp32 of odd width, without write gates, with an initial state that learns.
        dict(name="scan gradient odd", op="scan_grad", batch=5, tokens=1501, channels=333, type="f32", gtype="f32",
             gated=False, packed=True, initial=True),
        # One token of one sequence: latency.
        dict(name="scan token", op="scan_step", batch=1, tokens=1, channels=4096, type="bf16", gtype="bf16", gated=True),
        # One token of each of many sequences, their states scattered in a pool.
        dict(name="scan tokens batch", op="scan_step", batch=256, tokens=1, channels=4096, type="bf16", gtype="bf16",
             gated=True),
        # The log probability of a short answer: every weight of the output layer is read for a few tokens.
        dict(name="loss score", op="loss", tokens=48, vocabulary=65536, dim=4096, type="bf16", padded=False),
        # Loss and gradients of the output layer in a training step.
        dict(name="loss step", op="loss_grad", tokens=8192, vocabulary=65536, dim=2048, type="bf16", padded=False),
        # The same of a small model in fp32, odd in every size, some tokens without a target.
        dict(name="loss step odd", op="loss_grad", tokens=777, vocabulary=10007, dim=333, type="f32", padded=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "scan", "scan_grad", "scan_step", "loss", "loss_grad"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("embed", "embed_grad"):
        dim = rng.choice([_spread(rng, 16, 8192), 8 * _spread(rng, 8, 1024)])
        case = dict(op=op, tokens=_spread(rng, 1, max(2, min(65536, 33_000_000 // dim))),
                    vocabulary=_spread(rng, 16, max(32, min(200_000, 130_000_000 // dim))), dim=dim, type=kind,
                    padded=rng.random() < 0.4)
        if op == "embed_grad":
            case["added"] = rng.random() < 0.5
        return case
    if op in ("loss", "loss_grad"):
        dim = rng.choice([_spread(rng, 16, 4096), 8 * _spread(rng, 4, 512)])
        vocabulary = _spread(rng, 20, min(130_000, 270_000_000 // dim))
        most = min(16384, 500_000_000 // vocabulary, (400_000_000_000 if op == "loss" else 200_000_000_000)
                   // (vocabulary * dim))
        return dict(op=op, tokens=_spread(rng, 1, max(2, most)), vocabulary=vocabulary, dim=dim, type=kind,
                    padded=rng.random() < 0.5)
    channels = rng.choice([_spread(rng, 8, 8192), 8 * _spread(rng, 2, 1024)])
    case = dict(op=op, type=kind, gtype=rng.choice([kind, kind, "f32"]), gated=rng.random() < 0.6)
    if op == "scan_step":
        case.update(batch=_spread(rng, 1, max(2, min(1000, 2_000_000 // channels))), tokens=rng.choice([1, 1, 1, 2, 4]),
                    channels=channels)
        return case
    batch = _spread(rng, 1, 64)
    tokens = _spread(rng, 1, max(2, min(60_000, 66_000_000 // channels)))
    packed = rng.random() < 0.6
    if not packed:
        tokens = max(1, tokens // batch) * batch
    case.update(batch=batch, tokens=tokens, channels=channels, packed=packed, initial=rng.random() < 0.5)
    return case


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def tokens_of(count, vocabulary):
        """Tokens as a text has them, the r-th most frequent about 1 / r as often as the first; -1 is padding."""
        rank = torch.exp(uniform(count) * math.log(vocabulary)).long().clamp(1, vocabulary) - 1
        ids = torch.randperm(vocabulary, generator=gen, device="cuda")[rank]
        return torch.where(uniform(count) < 0.1, -1, ids) if case["padded"] else ids

    op, kind = case["op"], _TYPES[case["type"]]
    state = dict(case=case)
    if op in ("embed", "embed_grad"):
        count, vocabulary, dim = case["tokens"], case["vocabulary"], case["dim"]
        state["ids"] = tokens_of(count, vocabulary)
        state["scale"] = dim ** 0.5
        if op == "embed":
            state["table"] = (normal(vocabulary, dim) * dim ** -0.5).to(kind)
        else:
            state["dy"] = (normal(count, dim) * (0.2 + uniform(count, 1))).to(kind)
            if case["added"]:
                state["dtable"] = normal(vocabulary, dim).to(kind)
        return state
    if op in ("loss", "loss_grad"):
        count, vocabulary, dim = case["tokens"], case["vocabulary"], case["dim"]
        state["targets"] = tokens_of(count, vocabulary)
        w = 2 * dim ** -0.5 * normal(vocabulary, dim)
        state["w"] = w.to(kind)
        # Normalised activations that lean towards their target's weights: answers from a guess to a certainty.
        x = normal(count, dim) + 3 * uniform(count, 1) * w[state["targets"].clamp(min=0)]
        state["x"] = x.to(kind)
        if op == "loss_grad":  # the mean over tokens, weighted
            state["dloss"] = (0.5 + uniform(count)) / count
        return state
    batch, channels, gkind = case["batch"], case["channels"], _TYPES[case["gtype"]]
    lead = (batch, case["tokens"]) if op == "scan_step" else (case["tokens"],)
    state["x"] = normal(*lead, channels).to(kind)
    # Log decays from nearly none to a quick forgetting, by channel; write strengths between 0 and 1.
    rate = torch.logspace(-3, 0.5, channels, device="cuda")[torch.randperm(channels, generator=gen, device="cuda")]
    state["g"] = (-rate * torch.nn.functional.softplus(normal(*lead, channels))).to(gkind)
    state["beta"] = torch.sigmoid(normal(*lead, channels)).to(gkind) if case["gated"] else None
    if op == "scan_step":
        pool = batch + batch // 2
        state["pool"] = normal(pool, channels)
        state["slots"] = torch.randperm(pool, generator=gen, device="cuda")[:batch].int()
        return state
    lengths = _lengths(case)
    state["initial"] = normal(batch, channels) if case["initial"] else None
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    state["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if op == "scan_grad":
        state["dy"] = normal(*lead, channels).to(kind)
        state["dfinal"] = 0.5 * normal(batch, channels) if case["initial"] else None
        # What the forward call has returned.
        y, _ = _scan(state["x"], state["g"], state["beta"], state)
        state["y"] = y.to(kind)
    if case["packed"]:
        state["offsets"] = state["ends"]
    else:
        state["offsets"] = None
        for name in ("x", "g", "beta", "dy", "y"):
            if state.get(name) is not None:
                state[name] = state[name].reshape(batch, lengths[0], channels)
    return state


# ---- the plain forms --------------------------------------------------------------------------------

def _combine(a, h):
    """h_t = a_t h_{t-1} + h_t along the first axis, by doubling the distance."""
    step = 1
    while step < a.shape[0]:
        h = torch.cat([h[:step], torch.addcmul(h[step:], a[step:], h[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return h


def _scan(x, g, beta, state):
    """All sequences behind one another: the first token of each drops what was there before."""
    batch, channels = state["case"]["batch"], state["case"]["channels"]
    x, a = x.reshape(-1, channels).float(), g.reshape(-1, channels).float().exp()
    if beta is not None:
        x = x * beta.reshape(-1, channels).float()
    begin, end = state["ends"][:-1].long(), state["ends"][1:].long()
    there = end > begin
    first, initial = begin[there], state["initial"]
    if initial is not None:
        x = x.index_put((first,), x[first] + a[first] * initial[there])
    y = _combine(a.index_fill(0, first, 0), x)
    final = x.new_zeros(batch, channels) if initial is None else initial.clone()
    final[there] = y[end[there] - 1]
    return y, final


def _scan_grad_plain(state):
    case = state["case"]
    batch, channels = case["batch"], case["channels"]
    flat = {n: state[n].reshape(-1, channels).float() for n in ("x", "g", "dy", "y")}
    a, d = flat["g"].exp(), flat["dy"]
    begin, end = state["ends"][:-1].long(), state["ends"][1:].long()
    there = end > begin
    first, last = begin[there], end[there] - 1
    if state["dfinal"] is not None:
        d = d.index_put((last,), d[last] + state["dfinal"][there])
    # d_t += a_{t+1} d_{t+1}, from the end
    after = torch.cat([a[1:], a[:1]]).index_fill(0, last, 0)
    d = _combine(after.flip(0), d.flip(0)).flip(0)
    before = torch.cat([flat["y"][:1], flat["y"][:-1]])
    before = before.index_fill(0, first, 0) if state["initial"] is None else \
        before.index_put((first,), state["initial"][there])
    out = {"dg": (d * a * before).to(state["g"].dtype)}
    if state["beta"] is None:
        out["dx"] = d.to(state["x"].dtype)
    else:
        out["dx"] = (d * state["beta"].reshape(-1, channels).float()).to(state["x"].dtype)
        out["dbeta"] = (d * flat["x"]).to(state["beta"].dtype)
    out = {n: t.reshape(state["x"].shape) for n, t in out.items()}
    if state["initial"] is not None:
        dinitial = d.new_zeros(batch, channels) if state["dfinal"] is None else state["dfinal"].clone()
        dinitial[there] = a[first] * d[first]
        out["dinitial"] = dinitial
    return out


def _step_plain(state):
    case, pool, slots = state["case"], state["pool"], state["slots"].long()
    h, outs = pool[slots], []
    for t in range(case["tokens"]):
        x = state["x"][:, t].float()
        if state["beta"] is not None:
            x = x * state["beta"][:, t].float()
        h = state["g"][:, t].float().exp() * h + x
        outs.append(h)
    pool[slots] = h
    return {"y": torch.stack(outs, 1).to(state["x"].dtype), "pool": pool}


def _loss_plain(state):
    x, w, targets = state["x"].float(), state["w"].float(), state["targets"]
    there = targets >= 0
    at = targets.clamp(min=0)[:, None]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + (logits - top).exp().sum(1).log()
    loss = torch.where(there, lse - logits.gather(1, at)[:, 0], 0)
    out = {"loss": loss, "lse": lse}
    if state["case"]["op"] == "loss":
        return out
    d = (logits - lse[:, None]).exp()
    d.scatter_add_(1, at, d.new_full(at.shape, -1))
    d *= (state["dloss"] * there)[:, None]
    out["dx"] = (d @ w).to(state["x"].dtype)
    out["dw"] = (d.t() @ x).to(state["w"].dtype)
    return out


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "embed":
        rows = state["table"][state["ids"].clamp(min=0)].float() * state["scale"]
        return {"y": (rows * (state["ids"] >= 0)[:, None]).to(state["table"].dtype)}
    if op == "embed_grad":
        there = state["ids"] >= 0
        dy = state["dy"].float() * (state["scale"] * there)[:, None]
        dtable = dy.new_zeros(case["vocabulary"], case["dim"]).index_add_(0, state["ids"].clamp(min=0), dy)
        if case["added"]:
            state["dtable"].copy_(state["dtable"].float() + dtable)
            return {"dtable": state["dtable"]}
        return {"dtable": dtable.to(state["dy"].dtype)}
    if op in ("loss", "loss_grad"):
        return _loss_plain(state)
    if op == "scan_step":
        return _step_plain(state)
    if op == "scan_grad":
        return _scan_grad_plain(state)
    y, final = _scan(state["x"], state["g"], state["beta"], state)
    return {"y": y.to(state["x"].dtype).reshape(state["x"].shape), "final": final}


# ---- the library's ----------------------------------------------------------------------------------

def _run_own(state):
    import fft_convolution_gb300 as fg

    case = state["case"]
    op = case["op"]
    if op == "embed":
        return {"y": fg.embedding(state["ids"], state["table"], scale=state["scale"])}
    if op == "embed_grad":
        return {"dtable": fg.embedding_backward(state["dy"], state["ids"], case["vocabulary"], scale=state["scale"],
                                                add_to=state.get("dtable"))}
    if op in ("loss", "loss_grad"):
        x, w, targets = state["x"], state["w"], state["targets"]
        loss, lse = fg.linear_cross_entropy(x, w, targets)
        if op == "loss":
            return {"loss": loss, "lse": lse}
        dx, dw = fg.linear_cross_entropy_backward(state["dloss"], x, w, targets, lse)
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    x, g, beta = state["x"], state["g"], state["beta"]
    if op == "scan_step":
        y = fg.linear_recurrence_step(x, g, state["pool"], beta=beta, slots=state["slots"])
        return {"y": y, "pool": state["pool"]}
    if op == "scan":
        y, final = fg.linear_recurrence(x, g, beta, initial_state=state["initial"], offsets=state["offsets"])
        return {"y": y, "final": final}
    dx, dg, dbeta, dinitial = fg.linear_recurrence_backward(
        state["dy"], x, g, state["y"], beta=beta, initial_state=state["initial"], offsets=state["offsets"],
        dfinal_state=state["dfinal"])
    out = {"dg": dg, "dx": dx}
    if beta is not None:
        out["dbeta"] = dbeta
    if state["initial"] is not None:
        out["dinitial"] = dinitial
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- work -------------------------------------------------------------------------------------------

def work(case):
    size = 4 if case["type"] == "f32" else 2
    op = case["op"]
    if op in ("embed", "embed_grad"):
        count, table = case["tokens"], case["vocabulary"] * case["dim"] * size
        rows = count * case["dim"] * size
        if op == "embed":  # rows that come again are read once; in the mean those are few
            return dict(bytes=min(rows, table) + rows + 8 * count, flops=count * case["dim"])
        changed = 2 * min(rows, table) if case["added"] else table
        return dict(bytes=rows + changed + 8 * count, flops=2 * count * case["dim"])
    if op in ("loss", "loss_grad"):
        count, vocabulary, dim = case["tokens"], case["vocabulary"], case["dim"]
        both = (count + vocabulary) * dim * size
        if op == "loss":
            return dict(bytes=both + 16 * count, flops=2 * count * vocabulary * dim)
        return dict(bytes=2 * both + 20 * count, flops=6 * count * vocabulary * dim)
    gsize = 4 if case["gtype"] == "f32" else 2
    n = case["tokens"] * case["channels"] * (case["batch"] if op == "scan_step" else 1)
    gates = n * gsize * (2 if case["gated"] else 1)
    states = case["batch"] * case["channels"] * 4
    if op == "scan_step":
        return dict(bytes=2 * n * size + gates + 2 * states, flops=4 * n)
    if op == "scan":
        return dict(bytes=2 * n * size + gates + states * (2 if case["initial"] else 1), flops=4 * n)
    # in: dy, y, the gates, and x where beta needs it; out: dx and the gates' gradients
    return dict(bytes=(4 if case["gated"] else 3) * n * size + 2 * gates + (3 * states if case["initial"] else 0),
                flops=8 * n)


# ---- from the definitions, in 64 bits ------------------------------------------------------------------

def _exact_embed(case, state):
    ids, scale = state["ids"], float(state["scale"])
    there = (ids >= 0).nonzero()[:, 0]
    if case["op"] == "embed":
        y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        y[there] = scale * state["table"].double()[ids[there]]
        return {"y": y}
    # tokens in order of their row, running sums by row
    order = there[torch.sort(ids[there], stable=True)[1]]
    rows, counts = torch.unique_consecutive(ids[order], return_counts=True)
    sums = torch.segment_reduce(state["dy"][order].double() * scale, "sum", lengths=counts, axis=0)
    dtable = state["dtable"].double() if case["added"] else \
        torch.zeros(case["vocabulary"], case["dim"], dtype=torch.float64, device="cuda")
    dtable[rows] += sums
    return {"dtable": dtable}


def _exact_loss(case, state):
    x, w, targets = state["x"].double(), state["w"].double(), state["targets"]
    logits = torch.einsum("nd,vd->nv", x, w)
    lse = torch.logsumexp(logits, 1)
    there = (targets >= 0).nonzero()[:, 0]
    loss = torch.zeros_like(lse)
    loss[there] = lse[there] - logits[there, targets[there]]
    out = {"loss": loss, "lse": lse}
    if case["op"] == "loss":
        return out
    p = torch.softmax(logits, 1)
    del logits
    p[there, targets[there]] -= 1
    weight = torch.zeros_like(lse)
    weight[there] = state["dloss"].double()[there]
    p *= weight[:, None]
    out["dx"] = torch.einsum("nv,vd->nd", p, w)
    out["dw"] = torch.einsum("nv,nd->vd", p, x)
    return out


def _exact_scan(case, state):
    """One token of all sequences after the other, each from its own first row; one that has ended stands still."""
    batch, channels, lengths = case["batch"], case["channels"], _lengths(case)
    names = ["x", "g", "beta"] + (["dy", "y"] if case["op"] == "scan_grad" else [])
    flat = {n: state[n].reshape(-1, channels) for n in names if state[n] is not None}
    begin, length = state["ends"][:-1].long(), torch.tensor(lengths, device="cuda")
    h = torch.zeros(batch, channels, dtype=torch.float64, device="cuda")
    if state["initial"] is not None:
        h = state["initial"].double()
    if case["op"] == "scan":
        y = torch.zeros(case["tokens"], channels, dtype=torch.float64, device="cuda")
        for t in range(max(lengths)):
            live = (length > t).nonzero()[:, 0]
            at = begin[live] + t
            u = flat["x"][at].double()
            if "beta" in flat:
                u = flat["beta"][at].double() * u
            new = torch.exp(flat["g"][at].double()) * h[live] + u
            h[live] = new
            y[at] = new
        return {"y": y.reshape(state["x"].shape), "final": h}
    d = torch.zeros_like(h) if state["dfinal"] is None else state["dfinal"].double()
    out = {"d" + n: torch.zeros(case["tokens"], channels, dtype=torch.float64, device="cuda")
           for n in ("g", "x", "beta") if n in flat}
    for t in reversed(range(max(lengths))):
        live = (length > t).nonzero()[:, 0]
        at = begin[live] + t
        now = d[live] + flat["dy"][at].double()
        a = torch.exp(flat["g"][at].double())
        before = h[live] if t == 0 else flat["y"][at - 1].double()
        out["dg"][at] = now * a * before
        if "beta" in flat:
            out["dx"][at] = now * flat["beta"][at].double()
            out["dbeta"][at] = now * flat["x"][at].double()
        else:
            out["dx"][at] = now
        d[live] = a * now
    out = {n: v.reshape(state["x"].shape) for n, v in out.items()}
    if state["initial"] is not None:
        out["dinitial"] = d
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        return _exact_embed(case, state)
    if op in ("loss", "loss_grad"):
        return _exact_loss(case, state)
    if op in ("scan", "scan_grad"):
        return _exact_scan(case, state)
    pool, slots = state["pool"].double(), state["slots"].long()
    h, y = pool[slots], torch.zeros(state["x"].shape, dtype=torch.float64, device="cuda")
    for t in range(case["tokens"]):
        u = state["x"][:, t].double()
        if state["beta"] is not None:
            u = u * state["beta"][:, t].double()
        h = torch.exp(state["g"][:, t].double()) * h + u
        y[:, t] = h
    pool[slots] = h
    return {"y": y, "pool": pool}
