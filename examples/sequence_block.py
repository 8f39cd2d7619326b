"""One block of a sequence model on the library's operators: embedded tokens,
layer norm, a long causal convolution along time, the gated delta rule (or the
gated linear recurrence), the cross entropy of the output layer; trained with
clipped gradients, then run one token at a time from its states.

    python examples/sequence_block.py [--steps 120] [--tokens 64] [--mixer delta|recurrence]

The task is recall: a sequence of (key, value) token pairs, then keys whose
values have to be answered.  Prints the loss on the way and how far the
token-by-token run is from the whole-sequence one.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fft_convolution_gb300 as fg  # noqa: E402


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table):
        ctx.save_for_backward(tokens)
        ctx.rows = table.shape[0]
        return fg.embedding(tokens, table)

    @staticmethod
    def backward(ctx, dy):
        return None, fg.embedding_backward(dy, *ctx.saved_tensors, ctx.rows)


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = fg.layer_norm(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        return fg.layer_norm_backward(dy, *ctx.saved_tensors)


class LongConvolution(torch.autograd.Function):
    """y_t = sum_{j <= t} filter_j x_{t-j} for every row and channel of x
    [batch, time, channels], one filter for all (not learnt)."""

    @staticmethod
    def run(x, taps):
        rows = x.transpose(1, 2).reshape(-1, x.shape[1]).contiguous()
        y = fg.convolve(rows, taps)[:, : x.shape[1]]
        return y.reshape(x.shape[0], x.shape[2], x.shape[1]).transpose(1, 2).contiguous()

    @staticmethod
    def forward(ctx, x, taps):
        ctx.save_for_backward(taps)
        return LongConvolution.run(x, taps)

    @staticmethod
    def backward(ctx, dy):
        # dx_s = sum_{t >= s} filter_{t-s} dy_t: the same convolution, time reversed
        return LongConvolution.run(dy.flip(1), ctx.saved_tensors[0]).flip(1), None


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return fg.delta_rule(q, k, v, g, beta)

    @staticmethod
    def backward(ctx, do, dstate):
        return fg.delta_rule_backward(do, *ctx.saved_tensors, dfinal_state=dstate)[:5]


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, beta):
        y, state = fg.linear_recurrence(x, g, beta)
        ctx.save_for_backward(x, g, y, beta)
        return y, state

    @staticmethod
    def backward(ctx, dy, dstate):
        return fg.linear_recurrence_backward(dy, *ctx.saved_tensors, dfinal_state=dstate)[:3]


class LinearCrossEntropy(torch.autograd.Function):
    """Losses of x weight^T against targets, per token."""

    @staticmethod
    def forward(ctx, x, weight, targets):
        loss, lse = fg.linear_cross_entropy(x, weight, targets)
        ctx.save_for_backward(x, weight, targets, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        return *fg.linear_cross_entropy_backward(dloss, *ctx.saved_tensors), None


class Block:
    def __init__(self, tokens: int, width: int, heads: int, seed: int = 0, mixer: str = "delta"):
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=gen) * shape[0] ** -0.5
            return w.cuda().requires_grad_()

        self.heads, self.size, self.mixer = heads, width // heads, mixer
        self.embed = weight(tokens, width)
        self.norm_w = torch.ones(width, device="cuda", requires_grad=True)
        self.norm_b = torch.zeros(width, device="cuda", requires_grad=True)
        self.project = weight(width, 3 * width)
        self.gates = weight(width, 2 * (heads if mixer == "delta" else width))
        # one row per token, as its cross entropy reads it
        self.out = weight(width, tokens).detach().t().contiguous().requires_grad_()
        # a short look back: each token sees its predecessor, and a long decaying tail
        self.taps = 0.02 * 0.9 ** torch.arange(64, device="cuda", dtype=torch.float32)
        self.taps[:2] = torch.tensor([0.5, 1.0])

    def parameters(self):
        return [self.embed, self.norm_w, self.norm_b, self.project, self.gates, self.out]

    def mixed(self, h, x):
        """The mixer's inputs from the convolved (h) and the plain (x) activations: q, k, v, g, beta of the
        delta rule, x, g, beta of the recurrence."""
        lead = h.shape[:-1]
        if self.mixer == "recurrence":
            g, beta = (h @ self.gates).chunk(2, -1)
            value = x @ self.project.chunk(3, -1)[2]
            return value, -torch.nn.functional.softplus(g - 4), torch.sigmoid(beta)
        wq, wk, wv = self.project.chunk(3, -1)
        # a value is stored under the key before it: keys from h, values and queries from x
        q, k, v = (t.reshape(*lead, self.heads, self.size) for t in (x @ wq, h @ wk, x @ wv))
        unit = torch.nn.functional.normalize
        gates = (h @ self.gates).reshape(*lead, 2, self.heads)
        g = -0.02 * torch.nn.functional.softplus(gates[..., 0, :])
        return unit(q, dim=-1), unit(k, dim=-1), v, g.contiguous(), torch.sigmoid(gates[..., 1, :]).contiguous()

    def hidden(self, tokens):
        """What the output layer reads, and the mixer's state behind the last token."""
        x = LayerNorm.apply(Embedding.apply(tokens, self.embed), self.norm_w, self.norm_b)
        h = LongConvolution.apply(x, self.taps)
        if self.mixer == "recurrence":
            return Recurrence.apply(*self.mixed(h, x))
        o, state = DeltaRule.apply(*self.mixed(h, x))
        return o.flatten(-2), state

    def forward(self, tokens):
        o, state = self.hidden(tokens)
        return o @ self.out.t(), state

    def empty_states(self, count):
        shape = (self.size * self.heads,) if self.mixer == "recurrence" else (self.heads, self.size, self.size)
        return torch.zeros(count, *shape, device="cuda")

    @torch.no_grad()
    def decode(self, tokens, states, slots, history):
        """The logits of one more token per sequence; states (a pool) and history change."""
        x = fg.layer_norm(fg.embedding(tokens, self.embed)[:, None], self.norm_w, self.norm_b)[0]
        history[:] = torch.cat([x, history[:, :-1]], 1)
        h = torch.einsum("btc,t->bc", history, self.taps)[:, None]
        if self.mixer == "recurrence":
            value, g, beta = self.mixed(h, x)
            o = fg.linear_recurrence_step(value, g, states, beta=beta, slots=slots)
        else:
            o = fg.delta_rule_step(*self.mixed(h, x), states, slots=slots).flatten(-2)
        return o[:, 0] @ self.out.t()


def recall_batch(gen, batch, pairs, symbols):
    """Tokens k1 v1 k2 v2 ... then keys in another order, each followed by its value."""
    keys = torch.stack([torch.randperm(symbols, generator=gen)[:pairs] for _ in range(batch)])
    values = symbols + torch.randint(symbols, (batch, pairs), generator=gen)
    order = torch.stack([torch.randperm(pairs, generator=gen) for _ in range(batch)])
    again = torch.stack([keys.gather(1, order), values.gather(1, order)], -1).flatten(1)
    return torch.cat([torch.stack([keys, values], -1).flatten(1), again], 1).cuda(), 2 * pairs


def train(steps: int = 120, tokens: int = 64, batch: int = 16, width: int = 128, heads: int = 2,
          lr: float = 0.01, mixer: str = "delta", report=print):
    gen = torch.Generator().manual_seed(1)
    pairs, symbols = tokens // 4, 128
    block = Block(2 * symbols, width, heads, mixer=mixer)
    params = block.parameters()
    optimizer = torch.optim.Adam(params, lr=lr)
    losses = []
    for step in range(steps):
        data, asked = recall_batch(gen, batch, pairs, symbols)
        o, _ = block.hidden(data)
        # the value after each of the keys that come again
        loss = LinearCrossEntropy.apply(o[:, asked:-1:2], block.out, data[:, asked + 1::2]).mean()
        optimizer.zero_grad()
        loss.backward()
        norm = fg.clip_grad_norm([p.grad for p in params], 1.0)
        optimizer.step()
        losses.append(loss.item())
        if step % 20 == 0 or step == steps - 1:
            report(f"step {step:4d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.3f}")
    return block, losses


def decode_error(block, tokens: int = 96, batch: int = 3):
    """Largest difference of the logits, one token at a time against the whole sequence at once."""
    data, _ = recall_batch(torch.Generator().manual_seed(2), batch, tokens // 4, 128)
    with torch.no_grad():
        want, _ = block.forward(data)
    pool = block.empty_states(2 * batch)
    slots = torch.arange(batch, device="cuda", dtype=torch.int32) * 2 + 1
    history = torch.zeros(batch, block.taps.numel(), block.embed.shape[1], device="cuda")
    got = torch.stack([block.decode(data[:, t], pool, slots, history)
                       for t in range(data.shape[1])], 1)
    return float((got - want).abs().max() / want.abs().max())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=120)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--mixer", choices=("delta", "recurrence"), default="delta")
    args = ap.parse_args()
    trained, _ = train(args.steps, args.tokens, mixer=args.mixer)
    print(f"one token at a time: logits off by {decode_error(trained):.1e}")
