"""A KDA layer trained and then served with the library's operators:

    python examples/kda_layer.py            # trains, then decodes what it has learnt

layer norm -> projections -> gated delta-rule recurrence -> norm of each head -> projection, with
a residual connection.  Training runs kda_layer_norm_fwd/bwd and kda_chunk_fwd/bwd under autograd;
serving reads the prompt with kda_chunk_fwd, which returns the state, and goes on token by token
with kda_step.  The task is to repeat a sequence after having seen it once.
"""

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_intra_gb300 as kda  # noqa: E402

K = 128


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = kda.kda_layer_norm_fwd(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        dx, dweight, dbias = kda.kda_layer_norm_bwd(dy.contiguous(), *ctx.saved_tensors)
        return dx, dweight, dbias


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, gate, beta):
        o, _, saved = kda.kda_chunk_fwd(q, k, v, gate, beta, save=True)
        ctx.save_for_backward(q, k, v, gate, beta, saved)
        return o

    @staticmethod
    def backward(ctx, do):
        *inputs, saved = ctx.saved_tensors
        return kda.kda_chunk_bwd(*inputs, do.contiguous(), saved, gate_grads_fp32=True)[:5]


class Layer(torch.nn.Module):
    """width -> width over [B, T, width]; BF16 in the matrix products and the recurrence."""

    def __init__(self, width, heads, value_heads):
        super().__init__()
        self.H, self.HV = heads, value_heads
        self.norm_w = torch.nn.Parameter(torch.ones(width))
        self.norm_b = torch.nn.Parameter(torch.zeros(width))
        self.head_w = torch.nn.Parameter(torch.ones(K))
        self.head_b = torch.nn.Parameter(torch.zeros(K))
        sizes = [heads * K, heads * K, value_heads * K, value_heads * K, value_heads]
        self.sizes = sizes
        self.inp = torch.nn.Linear(width, sum(sizes), bias=False)
        self.out = torch.nn.Linear(value_heads * K, width, bias=False)
        # half-lives from a few to some thousand tokens, half the correction at first
        self.decay = torch.nn.Parameter(torch.linspace(-9, -2, K).repeat(value_heads, 1))

    def inputs(self, x):
        """q, k, v, gate, beta of [..., width] activations."""
        h = LayerNorm.apply(x, self.norm_w, self.norm_b)
        parts = F.linear(h, self.inp.weight.to(h.dtype)).split(self.sizes, -1)
        q, k, v, g = (p.unflatten(-1, (-1, K)) for p in parts[:4])
        q, k = (F.normalize(t.float(), dim=-1).to(x.dtype) for t in (q, k))
        gate = -F.softplus(g.float() + self.decay)
        return q, k, v.contiguous(), gate, parts[4].float().sigmoid()

    def outputs(self, x, o):
        o = LayerNorm.apply(o, self.head_w, self.head_b)
        return x + F.linear(o.flatten(-2), self.out.weight.to(o.dtype))

    def forward(self, x):
        return self.outputs(x, Recurrence.apply(*self.inputs(x)))

    @torch.no_grad()
    def prefill(self, x):
        """(outputs, state [B, HV, 128, 128]) of a prompt [B, T, width]."""
        o, state, _ = kda.kda_chunk_fwd(*self.inputs(x), output_final_state=True)
        return self.outputs(x, o), state

    @torch.no_grad()
    def step(self, x, state):
        """Outputs of one more token a sequence, x [B, width]; the state is updated in place."""
        return self.outputs(x, kda.kda_step(*self.inputs(x), state))


class Model(torch.nn.Module):
    def __init__(self, vocabulary, width, heads, value_heads, layers, layer=Layer):
        super().__init__()
        self.embed = torch.nn.Embedding(vocabulary, width)
        self.before = torch.nn.Embedding(vocabulary, width)  # of the token before
        torch.nn.init.normal_(self.embed.weight, std=width ** -0.5)
        torch.nn.init.normal_(self.before.weight, std=width ** -0.5)
        self.layers = torch.nn.ModuleList(
            [layer(width, heads, value_heads) for _ in range(layers)])
        self.norm_w = torch.nn.Parameter(torch.ones(width))
        self.norm_b = torch.nn.Parameter(torch.zeros(width))

    def inputs(self, tokens, before):
        return (self.embed(tokens) + self.before(before)).to(torch.bfloat16)

    def logits(self, x):
        x = LayerNorm.apply(x, self.norm_w, self.norm_b)
        return F.linear(x, self.embed.weight.to(x.dtype)).float()

    def forward(self, tokens):
        x = self.inputs(tokens, F.pad(tokens, (1, -1)))
        for layer in self.layers:
            x = layer(x)
        return self.logits(x)

    @torch.no_grad()
    def generate(self, prompt, count):
        """`count` tokens after the prompts [B, T], the likeliest each time."""
        x, states = self.inputs(prompt, F.pad(prompt, (1, -1))), []
        for layer in self.layers:
            x, state = layer.prefill(x)
            states.append(state)
        before, token = prompt[:, -1], self.logits(x[:, -1].contiguous()).argmax(-1)
        out = [token]
        while len(out) < count:
            x = self.inputs(token, before)
            for layer, state in zip(self.layers, states):
                x = layer.step(x, state)
            before, token = token, self.logits(x).argmax(-1)
            out.append(token)
        return torch.stack(out, 1)


def batch(n, length, vocabulary, gen):
    """[n, 2 length]: different tokens in random order, then the same again."""
    x = torch.rand(n, vocabulary, device="cuda", generator=gen).argsort(1)[:, :length]
    return torch.cat([x, x], 1)


def run(steps=200, sequences=32, length=32, vocabulary=64, width=256, heads=2, value_heads=4,
        layers=2, lr=2e-3, seed=0, verbose=True, layer=Layer):
    """Trains and serves; returns (first loss, last loss, share of repeated tokens right)."""
    torch.manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    model = Model(vocabulary, width, heads, value_heads, layers, layer).cuda()
    optim = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for i in range(steps):
        x = batch(sequences, length, vocabulary, gen)
        logits = model(x[:, :-1])[:, length - 1:]  # only the repetition can be foretold
        loss = F.cross_entropy(logits.flatten(0, 1), x[:, length:].flatten())
        optim.zero_grad()
        loss.backward()
        optim.step()
        losses.append(loss.item())
        if verbose and i % 50 == 0:
            print(f"step {i:4d}  loss {losses[-1]:.3f}")
    x = batch(sequences, length, vocabulary, gen)
    # the prompt ends with the repetition's first token: the rest is decoded
    got = model.generate(x[:, :length + 1], length - 1)
    right = (got == x[:, length + 1:]).float().mean().item()
    if verbose:
        print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; {100 * right:.1f}% of the tokens "
              f"repeated from the state alone")
    return losses[0], losses[-1], right


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    run(ap.parse_args().steps)
