"""Convolution, scan and matrix product at the ends of their range: sums beyond the 16-bit type, far
tails of a derivative, long memories, and what is left behind when a kernel gives up."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import BF, F64, HF, act64, cuda, make_linear, rel, tol

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


# ---------------------------------------------------------------------------- a wait that gives up
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N,pre", [
    (300, 520, 136, True),     # a few tiles, results by copies
    (130, 77, 129, True),      # rows on odd boundaries
    (40, 4096, 64, False),     # the contraction cut into parts
    (40000, 64, 264, False),   # several tiles a pair of blocks of threads
    (20000, 64, 521, True),    # ... on odd boundaries
    (5, 4096, 4000, False),    # few rows of a long contraction
])
def test_what_a_kernel_that_gives_up_leaves(M, K, N, pre, dtype):
    """Everything it had still to write is NaN, nothing is left as it was, and the next call is right."""
    x = make_linear(M, K, N, dtype, seed=M)
    c = cuda(x)
    act = "silu" if pre else None
    if N % 8 == 0 and K >= 64:
        y = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
        dx = torch.full((M, K), 3.0, dtype=dtype, device="cuda")
    else:
        y = dx = None
    saved0 = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"], activation="silu", save=True)[1]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    with kda.use_library(kda.DEBUG_LIB_PATH):
        kda.kda_debug_set_flags(word)
        kda.kda_debug_set_give_up(True)
        try:
            got, saved = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"], c["residual"], activation=act,
                                            save=pre, y=y)
            torch.cuda.synchronize()
            assert word.item() == 4  # KDA_DBG_WAIT alone
            gdx, gdw, gdb = kda.kda_linear_bwd(c["dy"], c["x"], c["weight"], saved0, activation="silu", dx=dx)
            torch.cuda.synchronize()
        finally:
            kda.kda_debug_set_give_up(False)
            kda.kda_debug_set_flags(None)
        assert word.item() == 4
        for name, t in (("y", got), ("saved", saved), ("dx", gdx), ("dweight", gdw)):
            assert t is None or torch.isnan(t).all(), name
        assert torch.isfinite(gdb).all()  # (of a kernel without such waits)
        want = x["x"].to(F64) @ x["weight"].to(F64).T + x["bias"].to(F64)
        again = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"], activation=None)[0]
        assert rel(again, want) <= tol(dtype)
    with pytest.raises(kda.KdaError):
        kda.kda_debug_set_give_up(True)  # not in the normal build
