"""One block of a sequence model on the library's operators: layer norm, a long
causal convolution along time, the gated delta rule; trained with clipped
gradients, then run one token at a time from its states.

    python examples/sequence_block.py [--steps 120] [--tokens 64]

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


class Block:
    def __init__(self, tokens: int, width: int, heads: int, seed: int = 0):
        gen = torch.Generator().manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=gen) * shape[0] ** -0.5
            return w.cuda().requires_grad_()

        self.heads, self.size = heads, width // heads
        self.embed = weight(tokens, width)
        self.norm_w = torch.ones(width, device="cuda", requires_grad=True)
        self.norm_b = torch.zeros(width, device="cuda", requires_grad=True)
        self.project = weight(width, 3 * width)
        self.gates = weight(width, 2 * heads)
        self.out = weight(width, tokens)
        # a short look back: each token sees its predecessor, and a long decaying tail
        self.taps = 0.02 * 0.9 ** torch.arange(64, device="cuda", dtype=torch.float32)
        self.taps[:2] = torch.tensor([0.5, 1.0])

    def parameters(self):
        return [self.embed, self.norm_w, self.norm_b, self.project, self.gates, self.out]

    def mixed(self, h, x):
        """q, k, v, g, beta from the convolved (h) and the plain (x) activations."""
        lead = h.shape[:-1]
        wq, wk, wv = self.project.chunk(3, -1)
        # a value is stored under the key before it: keys from h, values and queries from x
        q, k, v = (t.reshape(*lead, self.heads, self.size) for t in (x @ wq, h @ wk, x @ wv))
        unit = torch.nn.functional.normalize
        gates = (h @ self.gates).reshape(*lead, 2, self.heads)
        g = -0.02 * torch.nn.functional.softplus(gates[..., 0, :])
        return unit(q, dim=-1), unit(k, dim=-1), v, g, torch.sigmoid(gates[..., 1, :])

    def forward(self, tokens):
        x = LayerNorm.apply(self.embed[tokens], self.norm_w, self.norm_b)
        h = LongConvolution.apply(x, self.taps)
        q, k, v, g, beta = self.mixed(h, x)
        o, state = DeltaRule.apply(q, k, v, g.contiguous(), beta.contiguous())
        return o.flatten(-2) @ self.out, state

    @torch.no_grad()
    def decode(self, tokens, states, slots, history):
        """The logits of one more token per sequence; states (a pool) and history change."""
        x = fg.layer_norm(self.embed[tokens][:, None], self.norm_w, self.norm_b)[0]
        history[:] = torch.cat([x, history[:, :-1]], 1)
        h = torch.einsum("btc,t->bc", history, self.taps)[:, None]
        q, k, v, g, beta = self.mixed(h, x)
        o = fg.delta_rule_step(q, k, v, g.contiguous(), beta.contiguous(), states, slots=slots)
        return o.flatten(-2)[:, 0] @ self.out


def recall_batch(gen, batch, pairs, symbols):
    """Tokens k1 v1 k2 v2 ... then keys in another order, each followed by its value."""
    keys = torch.stack([torch.randperm(symbols, generator=gen)[:pairs] for _ in range(batch)])
    values = symbols + torch.randint(symbols, (batch, pairs), generator=gen)
    order = torch.stack([torch.randperm(pairs, generator=gen) for _ in range(batch)])
    again = torch.stack([keys.gather(1, order), values.gather(1, order)], -1).flatten(1)
    return torch.cat([torch.stack([keys, values], -1).flatten(1), again], 1).cuda(), 2 * pairs


def train(steps: int = 120, tokens: int = 64, batch: int = 16, width: int = 128, heads: int = 2,
          lr: float = 0.01, report=print):
    gen = torch.Generator().manual_seed(1)
    pairs, symbols = tokens // 4, 128
    block = Block(2 * symbols, width, heads)
    params = block.parameters()
    optimizer = torch.optim.Adam(params, lr=lr)
    losses = []
    for step in range(steps):
        data, asked = recall_batch(gen, batch, pairs, symbols)
        logits, _ = block.forward(data)
        # the value after each of the keys that come again
        loss = torch.nn.functional.cross_entropy(logits[:, asked:-1:2].flatten(0, 1),
                                                 data[:, asked + 1::2].flatten())
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
    pool = torch.zeros(2 * batch, block.heads, block.size, block.size, device="cuda")
    slots = torch.arange(batch, device="cuda", dtype=torch.int32) * 2 + 1
    history = torch.zeros(batch, block.taps.numel(), block.embed.shape[1], device="cuda")
    got = torch.stack([block.decode(data[:, t], pool, slots, history)
                       for t in range(data.shape[1])], 1)
    return float((got - want).abs().max() / want.abs().max())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=120)
    ap.add_argument("--tokens", type=int, default=64)
    args = ap.parse_args()
    trained, _ = train(args.steps, args.tokens)
    print(f"one token at a time: logits off by {decode_error(trained):.1e}")
