"""The language model of kda_layer.py with a selective scan in place of the delta rule:

    python examples/scan_layer.py            # trains, then decodes what it has learnt

layer norm -> projection -> short convolution -> scan, whose step sizes and vectors are projections
of the convolution's result -> projection, with the residual in its epilogue.  Training runs
kda_linear_fwd/bwd, kda_conv_fwd/bwd and kda_scan_fwd/bwd under autograd; serving reads the prompt with
the same calls, which return the states, and goes on with kda_conv_step and kda_scan_step.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import kda_layer  # noqa: E402

kda = kda_layer.kda


class Linear(torch.autograd.Function):
    """x weight^T (+ residual)."""

    @staticmethod
    def forward(ctx, x, weight, residual=None):
        ctx.save_for_backward(x, weight)
        ctx.more = residual is not None
        return kda.kda_linear_fwd(x, weight, residual=residual)[0]

    @staticmethod
    def backward(ctx, dy):
        dy = dy.contiguous()
        dx, dweight, _ = kda.kda_linear_bwd(dy, *ctx.saved_tensors, bias_grad=False)
        return dx, dweight, dy if ctx.more else None


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return kda.kda_conv_fwd(x, weight, bias, activation="silu")[0]

    @staticmethod
    def backward(ctx, dy):
        return kda.kda_conv_bwd(dy.contiguous(), *ctx.saved_tensors, activation="silu")[:3]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, delta, A, B, C, D, z, delta_bias):
        y, _, saved = kda.kda_scan_fwd(u, delta, A, B, C, D, z, delta_bias, save=True)
        ctx.save_for_backward(u, delta, A, B, C, saved, D, z, delta_bias)
        return y

    @staticmethod
    def backward(ctx, dy):
        return kda.kda_scan_bwd(dy.contiguous(), *ctx.saved_tensors)[:8]


class ScanLayer(torch.nn.Module):
    """width -> width over [B, T, width]; 16-bit activations, parameters and states in FP32."""

    def __init__(self, width, inner=None, states=16, taps=4):
        super().__init__()
        inner = inner or 2 * width
        rank = -(-width // 16)
        self.sizes = [rank, states, states]

        def matrix(out, of):
            return torch.nn.Parameter(torch.randn(out, of) * of ** -0.5)

        self.norm_w = torch.nn.Parameter(torch.ones(width))
        self.norm_b = torch.nn.Parameter(torch.zeros(width))
        self.inp, self.out = matrix(2 * inner, width), matrix(width, inner)
        self.conv_w, self.conv_b = matrix(inner, taps), torch.nn.Parameter(torch.zeros(inner))
        self.select, self.delta = matrix(sum(self.sizes), inner), matrix(inner, rank)
        # step sizes from 0.001 to 0.1 at first, state n fading n times as fast
        at = torch.exp(torch.empty(inner).uniform_(math.log(1e-3), math.log(1e-1)))
        self.delta_bias = torch.nn.Parameter(at + torch.log(-torch.expm1(-at)))
        self.log_A = torch.nn.Parameter(torch.arange(1, states + 1).float().log().repeat(inner, 1))
        self.skip = torch.nn.Parameter(torch.ones(inner))

    def before(self, x):
        """What the convolution reads, and the gate."""
        h = kda_layer.LayerNorm.apply(x, self.norm_w, self.norm_b)
        return Linear.apply(h, self.inp.to(x.dtype)).chunk(2, -1)

    def scan_inputs(self, u, z):
        d, B, C = Linear.apply(u, self.select.to(u.dtype)).split(self.sizes, -1)
        delta = Linear.apply(d, self.delta.to(u.dtype))
        return (u, delta, -self.log_A.exp(), B.unsqueeze(-2), C.unsqueeze(-2)), (self.skip, z, self.delta_bias)

    def after(self, x, y):
        return Linear.apply(y, self.out.to(x.dtype), x)

    def forward(self, x):
        v, z = self.before(x)
        ins, more = self.scan_inputs(Conv.apply(v, self.conv_w, self.conv_b), z)
        return self.after(x, Scan.apply(*ins, *more))

    @torch.no_grad()
    def prefill(self, x):
        """(outputs, states of convolution and scan) of a prompt [B, T, width]."""
        v, z = self.before(x)
        u, inputs = kda.kda_conv_fwd(v, self.conv_w, self.conv_b, activation="silu", output_final_state=True)
        ins, more = self.scan_inputs(u, z)
        y, state, _ = kda.kda_scan_fwd(*ins, *more, output_final_state=True)
        return self.after(x, y), (inputs, state)

    @torch.no_grad()
    def step(self, x, states):
        """Outputs of one more token a sequence, x [B, width]; the states are updated in place."""
        v, z = self.before(x)
        ins, more = self.scan_inputs(
            kda.kda_conv_step(v, states[0], self.conv_w, self.conv_b, activation="silu"), z)
        return self.after(x, kda.kda_scan_step(*ins, states[1], *more))


def run(steps=300, length=8, vocabulary=16, **kw):
    """(Shorter sequences than kda_layer.py's: this state holds on to fewer tokens.)"""
    return kda_layer.run(steps, length=length, vocabulary=vocabulary,
                         layer=lambda width, heads, value_heads: ScanLayer(width), **kw)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=300)
    run(ap.parse_args().steps)
