"""The operators of a small recurrent language model together, as a training
step and a decoding loop use them: embedded tokens, layer norm, the linear
recurrence, the loss of an output layer that shares the embedding's table, and
the clipped gradients; against the same model in 64-bit torch.

Tolerances, fixed before the first run: fp32 operators of errors of a few 2^-24
each, relative to what they sum, through four layers and sums of up to a
thousand terms: 2e-5 of a tensor's 2-norm.  With bfloat16 activations every layer
rounds by 2^-8 at most and passes on the errors of those before it with a gain
near 1: 8 layers forward and back, 2^-5."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg(fg_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return fg_lib


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sequence_block.py")
    spec = importlib.util.spec_from_file_location("sequence_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def made(seed, kind, batch=3, time=70, words=301, width=96):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    data = torch.randint(words, (batch, time + 1), generator=gen, device="cuda")
    tokens, targets = data[:, :-1].clone(), data[:, 1:].clone()
    tokens[0, 50:] = -1      # a padded sequence
    targets[0, 49:] = -100
    p = dict(table=normal(words, width) * width ** -0.5, w=1 + 0.1 * normal(width), b=0.1 * normal(width),
             g=-torch.nn.functional.softplus(normal(batch, time, width) - 2), beta=torch.sigmoid(normal(batch, time, width)))
    return tokens, targets, {n: t.to(kind) for n, t in p.items()}


def step64(tokens, targets, p, scale):
    q = {n: t.double().requires_grad_() for n, t in p.items()}
    x = scale * torch.where(tokens[..., None] >= 0, q["table"][tokens.clamp(min=0)], 0)
    mu = x.mean(-1, keepdim=True)
    y = (x - mu) / ((x - mu).square().mean(-1, keepdim=True) + 1e-5).sqrt() * q["w"] + q["b"]
    h, rows = y.new_zeros(y.shape[0], y.shape[2]), []
    for t in range(y.shape[1]):
        h = q["g"][:, t].exp() * h + q["beta"][:, t] * y[:, t]
        rows.append(h)
    logits = torch.stack(rows, 1) @ q["table"].t()
    there = targets >= 0
    each = torch.logsumexp(logits, -1) - logits.gather(-1, targets.clamp(min=0)[..., None])[..., 0]
    loss = (each * there).sum() / there.sum()
    names = list(q)
    return loss, dict(zip(names, torch.autograd.grad(loss, [q[n] for n in names]))), h


def step(fg, tokens, targets, p, scale):
    x = fg.embedding(tokens, p["table"], scale=scale)
    y, mean, rstd = fg.layer_norm(x, p["w"], p["b"])
    h, last = fg.linear_recurrence(y, p["g"], p["beta"])
    loss, lse = fg.linear_cross_entropy(h, p["table"], targets)
    count = (targets >= 0).sum()
    dloss = (1 / count).float().expand(targets.shape)
    dh, dtable = fg.linear_cross_entropy_backward(dloss, h, p["table"], targets, lse)
    dy, dg, dbeta, _ = fg.linear_recurrence_backward(dh, y, p["g"], h, beta=p["beta"])
    dx, dw, db = fg.layer_norm_backward(dy, x, p["w"], mean, rstd)
    fg.embedding_backward(dx, tokens, p["table"].shape[0], scale=scale, add_to=dtable)
    return loss.sum() / count, dict(table=dtable, w=dw, b=db, g=dg, beta=dbeta), last


@pytest.mark.parametrize("kind,tol", [(torch.float32, 2e-5), (torch.bfloat16, 2.0 ** -5)])
def test_training_step(fg, kind, tol):
    tokens, targets, p = made(1, kind)
    loss, grads, last = step(fg, tokens, targets, p, 5.0)
    want, exact, last64 = step64(tokens, targets, p, 5.0)
    assert abs(float(loss - want)) <= tol * float(want)
    assert rel(last, last64.detach()) <= tol
    for name, t in grads.items():
        assert t.dtype == kind and rel(t, exact[name]) <= tol, name
    total = torch.cat([t.double().flatten() for t in exact.values()]).norm()
    norm = fg.clip_grad_norm(list(grads.values()), 0.5 * float(total))
    assert abs(float(norm) / float(total) - 1) <= tol
    for name, t in grads.items():
        assert rel(t, exact[name] / 2) <= 2 * tol, name


def test_captured_training_step(fg):
    tokens, targets, p = made(2, torch.float32)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(fg, tokens, targets, p, 5.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads, last = step(fg, tokens, targets, p, 5.0)
    for seed in (3, 4):
        t2, y2, p2 = made(seed, torch.float32)
        tokens.copy_(t2)
        targets.copy_(y2)
        for n in p:
            p[n].copy_(p2[n])
        graph.replay()
        again, g2, l2 = step(fg, tokens, targets, p, 5.0)
        assert torch.equal(loss, again) and torch.equal(last, l2)
        assert all(torch.equal(grads[n], g2[n]) for n in grads)


def test_decoding_scores_what_was_trained_on(fg):
    # token by token from stored states: the losses of the whole sequence
    tokens, targets, p = made(5, torch.float32)
    x = fg.embedding(tokens, p["table"], scale=5.0)
    y = fg.layer_norm(x, p["w"], p["b"])[0]
    h, _ = fg.linear_recurrence(y, p["g"], p["beta"])
    want, _ = fg.linear_cross_entropy(h, p["table"], targets)
    pool = torch.zeros(7, 96, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    for t in range(tokens.shape[1]):
        one = slice(t, t + 1)
        y = fg.layer_norm(fg.embedding(tokens[:, one], p["table"], scale=5.0), p["w"], p["b"])[0]
        o = fg.linear_recurrence_step(y, p["g"][:, one], pool, beta=p["beta"][:, one], slots=slots)
        loss, _ = fg.linear_cross_entropy(o, p["table"], targets[:, one])
        assert (loss - want[:, one]).abs().max() <= 1e-4
    assert not pool[[1, 2, 3, 5]].any()


def test_autograd_notices_tensors_changed_in_place(fg):
    def raises(shape, change):
        a = torch.ones(*shape, device="cuda", requires_grad=True)
        kept = a * 1.0
        y = (kept * kept).sum()
        change(kept.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    ids = torch.tensor([1, 0], device="cuda")
    x = torch.ones(2, 3, 8, device="cuda")
    raises((2, 8), lambda t: fg.embedding(ids, torch.ones(2, 8, device="cuda"), out=t))
    raises((2, 8), lambda t: fg.embedding_backward(torch.ones(2, 8, device="cuda"), ids, 2, add_to=t))
    raises((2, 3, 8), lambda t: fg.linear_recurrence(x, -x, out=t))
    raises((2, 8), lambda t: fg.linear_recurrence_step(x, -x, t))
    raises((2, 3, 8), lambda t: fg.linear_recurrence_step(x, -x, torch.zeros(2, 8, device="cuda"), out=t))


def test_copies_belong_to_the_calls_stream(fg):
    # strided inputs on a side stream, while the current one is busy with work that does not touch them
    wide = torch.randn(64, 400, device="cuda")
    table, ids, targets = torch.randn(80, 100, device="cuda")[:, ::2], torch.arange(64, device="cuda"), torch.arange(64, device="cuda")
    x = wide[:, :100:2]
    call = lambda **kw: (fg.embedding(ids, table, **kw), fg.embedding_backward(x, ids, 80, **kw),  # noqa: E731
                         *fg.linear_recurrence(x[None], -x[None].abs(), **kw), *fg.linear_cross_entropy(x, table, targets, **kw))
    want = call()
    busy, side = torch.randn(8192, 8192, device="cuda"), torch.cuda.Stream()
    gates = -x[None].abs()
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(8):
            busy @ busy
        got = (fg.embedding(ids, table, stream=side), fg.embedding_backward(x, ids, 80, stream=side),
               *fg.linear_recurrence(x[None], gates, stream=side), *fg.linear_cross_entropy(x, table, targets, stream=side))
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        torch.cuda.synchronize()


@pytest.mark.parametrize("mixer", ["delta", "recurrence"])
def test_the_examples_gradients(fg, mixer):
    # against the same block of plain torch operations in 64 bits
    module = example()
    block = module.Block(64, 32, 2, mixer=mixer)
    data = torch.randint(64, (3, 40), generator=torch.Generator().manual_seed(1)).cuda()
    o, _ = block.hidden(data)
    module.LinearCrossEntropy.apply(o[:, :-1], block.out, data[:, 1:]).mean().backward()
    got = [p.grad.double() for p in block.parameters()]
    params = [p.detach().double().requires_grad_() for p in block.parameters()]
    embed, norm_w, norm_b, project, gates, out = params
    x = embed[data]
    x = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt() * norm_w + norm_b
    taps = block.taps.double()
    h = sum(taps[j] * torch.nn.functional.pad(x, (0, 0, j, 0))[:, : x.shape[1]] for j in range(min(len(taps), x.shape[1])))
    twin = module.Block(64, 32, 2, mixer=mixer)
    twin.project, twin.gates = project, gates
    state, rows = 0, []
    if mixer == "recurrence":
        value, g, beta = twin.mixed(h, x)
        for t in range(40):
            state = g[:, t].exp() * state + beta[:, t] * value[:, t]
            rows.append(state)
    else:
        q, k, v, g, beta = twin.mixed(h, x)
        state = q.new_zeros(3, 2, 16, 16)
        for t in range(40):
            state = state * g[:, t].exp()[..., None, None]
            u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", state, k[:, t]))
            state = state + k[:, t, :, :, None] * u[:, :, None]
            rows.append(torch.einsum("bhkv,bhk->bhv", state, q[:, t]).flatten(1) * 16 ** -0.5)
    logits = torch.stack(rows, 1)[:, :-1] @ out.t()
    torch.nn.functional.cross_entropy(logits.flatten(0, 1), data[:, 1:].flatten()).backward()
    for p, mine in zip(params, got):
        if p.grad is None:  # the recurrence takes a third of the projection
            continue
        assert float((mine - p.grad).norm()) <= 1e-4 * float(p.grad.norm())


def test_the_example_decodes_with_the_recurrence(fg):
    module = example()
    block, losses = module.train(steps=3, tokens=32, mixer="recurrence", report=lambda line: None)
    assert all(x == x for x in losses)
    assert module.decode_error(block, tokens=48) <= 1e-4
