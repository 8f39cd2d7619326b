"""The gated delta rule token by token in 64 bits on the CPU: the recurrence
itself and, for its gradients, the same recurrence run backwards."""
import torch


def unit(t):
    return t / t.norm(dim=-1, keepdim=True)


def inputs(seed, batch, tokens, kheads, vheads, dk, dv, kind=torch.float32):
    """q, k, v, g, beta as [batch, tokens, heads, ...] (CPU): unit keys and
    queries, decays from slow to quick by head."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    q = unit(normal(batch, tokens, kheads, dk)).to(kind)
    k = unit(normal(batch, tokens, kheads, dk) + 0.5 * normal(1, 1, kheads, dk)).to(kind)
    v = normal(batch, tokens, vheads, dv).to(kind)
    rate = torch.logspace(-2, 0.3, vheads, dtype=torch.float64)
    g = (-rate * torch.nn.functional.softplus(normal(batch, tokens, vheads))).float()
    beta = torch.sigmoid(normal(batch, tokens, vheads)).float()
    return q, k, v, g, beta


def forward(q, k, v, g, beta, scale=None, state=None):
    """(o, final state) of [tokens, heads, ...] inputs of one sequence."""
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    group = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    s = torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if state is None \
        else state.double()
    outs = []
    for t in range(q.shape[0]):
        s = s * g[t].exp()[:, None, None]
        u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", s, k[t]))
        s = s + k[t][:, :, None] * u[:, None, :]
        outs.append(scale * torch.einsum("hkv,hk->hv", s, q[t]))
    return (torch.stack(outs) if outs else v.new_zeros(v.shape)), s


def backward(do, q, k, v, g, beta, scale=None, state=None, dfinal=None):
    """(dq, dk, dv, dg, dbeta, dstate) for one sequence."""
    q, k, v, g, beta, do = (t.double() for t in (q, k, v, g, beta, do))
    heads, group = v.shape[1], v.shape[1] // q.shape[1]
    qe, ke = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    s = torch.zeros(heads, q.shape[2], v.shape[2], dtype=torch.float64) if state is None \
        else state.double()
    d = torch.zeros_like(s) if dfinal is None else dfinal.double()
    keep = []
    for t in range(q.shape[0]):
        before = s * g[t].exp()[:, None, None]
        miss = v[t] - torch.einsum("hkv,hk->hv", before, ke[t])
        s = before + ke[t][:, :, None] * (beta[t][:, None] * miss)[:, None, :]
        keep.append((before, miss, s))
    dq, dk, dv, dg, dbeta = (torch.zeros_like(t) for t in (qe, ke, v, g, beta))
    for t in reversed(range(q.shape[0])):
        before, miss, after = keep[t]
        dq[t] = scale * torch.einsum("hkv,hv->hk", after, do[t])
        d = d + scale * qe[t][:, :, None] * do[t][:, None, :]
        du = torch.einsum("hkv,hk->hv", d, ke[t])
        dy = beta[t][:, None] * du
        dk[t] = torch.einsum("hkv,hv->hk", d, beta[t][:, None] * miss) - \
            torch.einsum("hkv,hv->hk", before, dy)
        dv[t], dbeta[t] = dy, (du * miss).sum(-1)
        d = d - ke[t][:, :, None] * dy[:, None, :]
        dg[t] = (d * before).sum((-1, -2))
        d = d * g[t].exp()[:, None, None]

    def shared(t):
        return t.reshape(t.shape[0], heads // group, group, t.shape[2]).sum(2)

    return shared(dq), shared(dk), dv, dg, dbeta, d
