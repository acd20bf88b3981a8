"""Convolution, scan and matrix product at the ends of their range: sums beyond the 16-bit type, far
tails of a derivative, long memories, and what is left behind when a kernel gives up."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import BF, F64, HF, act64

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- sums beyond FP16
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,N", [(2, 12), (40, 13), (300, 16)])
def test_gradients_where_the_saved_sum_is_infinite(M, N, act):
    """x weight^T is +-70000 in two columns: infinite in FP16, where the derivative is 1 and 0."""
    gen = torch.Generator().manual_seed(M)
    x = torch.full((M, 8), 100.0, dtype=HF)
    w = (torch.randn(N, 8, generator=gen) / 100).to(HF)
    w[1], w[2] = 87.5, -87.5
    bias = torch.randn(N, generator=gen).to(HF)
    dy = torch.randn(M, N, generator=gen).to(HF)
    c = [t.cuda() for t in (x, w, bias, dy)]
    y, saved = kda.kda_linear_fwd(*c[:3], activation=act, save=True)
    assert torch.isposinf(saved[:, 1]).all() and torch.isneginf(saved[:, 2]).all()
    assert (y[:, 2] == 0).all()
    grads = kda.kda_linear_bwd(c[3], *c[:2], saved, activation=act)
    leaf = [t.to(F64).requires_grad_() for t in (x, w, bias)]
    want = torch.autograd.grad(act64(leaf[0] @ leaf[1].T + leaf[2], act), leaf, dy.to(F64))
    # relative to what an element's sum is made of: the derivative's place, dpre and the result are each
    # rounded to FP16 (2^-11), and the derivative changes by at most its place's rounding |pre| 2^-11,
    # |pre| < 8 in the finite columns; 1e-5 for FP32's own
    d = dy.to(F64).abs()
    size = (d @ w.to(F64).abs(), d.T @ x.to(F64).abs(), d.sum(0))
    for name, got, ref, s in zip(("dx", "dweight", "dbias"), grads, want, size):
        got = got.cpu().to(F64)
        assert torch.isfinite(got).all(), name
        assert ((got - ref).abs() <= s * (10 * 2.0 ** -11 + 1e-5) + 2.0 ** -24).all(), name
