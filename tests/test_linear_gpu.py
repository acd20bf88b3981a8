"""kda_linear_fwd and kda_linear_bwd against the definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import BF, F64, HF, SUMS, UNIT, act64, leaves, make_linear, rel

pytestmark = pytest.mark.gpu


def check(x, act=None, bias=True, residual=True, want_bias=True):
    names = ["x", "weight"] + ["bias"] * bias
    h = leaves(x, names)
    pre = h["x"] @ h["weight"].T
    if bias:
        pre = pre + h["bias"]
    want = act64(pre, act)
    if residual:
        want = want + x["residual"].to(F64)
    grads = dict(zip(names, torch.autograd.grad(want, [h[n] for n in names], x["dy"].to(F64))))
    c = {n: t.cuda() for n, t in x.items()}
    y, saved = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"] if bias else None,
                                  c["residual"] if residual else None, activation=act, save=True)
    dx, dw, db = kda.kda_linear_bwd(c["dy"], c["x"], c["weight"], saved, activation=act, bias_grad=bias)
    u = UNIT[x["x"].dtype]
    assert rel(y, want) <= u + SUMS, rel(y, want)
    # the gradients: saved and dpre are rounded once each (with slopes of at most 1.13 and their own
    # slopes of at most 0.8 beside values of a few units), then the result
    inner = 0 if act is None else 4 * u
    assert rel(dx, grads["x"]) <= u + inner + SUMS, rel(dx, grads["x"])
    assert rel(dw, grads["weight"]) <= u + inner + SUMS, rel(dw, grads["weight"])
    if bias:
        assert rel(db, grads["bias"]) <= u + inner + SUMS, rel(db, grads["bias"])
    if act is not None:
        assert rel(saved, pre) <= u + SUMS


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N", [(128, 64, 64), (128, 64, 128), (256, 128, 256), (1, 8, 8), (17, 72, 40),
                                   (129, 200, 264), (300, 520, 136), (64, 1000, 24), (200, 8, 520)])
def test_products(M, K, N, dtype):
    check(make_linear(M, K, N, dtype, seed=M + K), bias=False, residual=False)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", [None, "silu", "gelu", "relu"])
@pytest.mark.parametrize("M,K,N", [(3, 64, 80), (40, 96, 72), (150, 136, 200)])
def test_epilogues(M, K, N, act, dtype):
    x = make_linear(M, K, N, dtype, seed=M)
    check(x, act)
    check(x, act, bias=False)
    check(x, act, residual=False)


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (5, 7, 3), (31, 33, 65), (130, 77, 129), (257, 130, 190),
                                   (20, 1111, 1540)])
def test_sizes_that_are_a_multiple_of_nothing(M, K, N):
    check(make_linear(M, K, N, HF, seed=N), "silu")
    check(make_linear(M, K, N, BF, seed=N), None, bias=False)


@pytest.mark.parametrize("M", list(range(1, 21)) + [32, 33])
def test_few_rows(M):
    check(make_linear(M, 648, 152, BF, seed=M), "gelu")


@pytest.mark.parametrize("M,K,N", [(40, 4096, 64), (128, 8192, 128), (2500, 64, 72), (5000, 40, 16)])
def test_long_contractions(M, K, N):
    """Few tiles of the result: the contraction is cut and joined (of the weight's gradient, over M)."""
    check(make_linear(M, K, N, BF, seed=K), "silu")


@pytest.mark.parametrize("M,K,N", [(2048, 256, 2560), (3000, 512, 4104)])
def test_many_tiles(M, K, N):
    """Several tiles a CTA: both accumulators and every stage come round again."""
    check(make_linear(M, K, N, BF, seed=1), "silu")


def test_leading_dimensions():
    check(make_linear(0, 64, 72, BF, lead=(2, 3, 5)), "silu")
    check(make_linear(0, 64, 72, BF, lead=()), "relu")


@pytest.mark.parametrize("M", [6, 100])
@pytest.mark.parametrize("off", [0, 8, 3])
def test_slices_of_wider_tensors(off, M):
    K, N = 72, 88
    x = make_linear(M, K, N, BF, seed=off)
    c = {}
    for n in ("x", "weight", "residual", "dy"):
        w = torch.full((x[n].shape[0], x[n].shape[1] + off + 16), float("nan"), dtype=BF, device="cuda")
        c[n] = w[:, off:off + x[n].shape[1]]
        c[n].copy_(x[n])
    yw, dxw = (torch.full((M, w + 24), 7.0, dtype=BF, device="cuda") for w in (N, K))
    y, saved = kda.kda_linear_fwd(c["x"], c["weight"], x["bias"].cuda(), c["residual"], activation="silu",
                                  save=True, y=yw[:, off:off + N])
    dx, dw, db = kda.kda_linear_bwd(c["dy"], c["x"], c["weight"], saved, activation="silu",
                                    dx=dxw[:, off:off + K])
    h = leaves(x, ("x", "weight", "bias"))
    want = act64(h["x"] @ h["weight"].T + h["bias"], "silu") + x["residual"].to(F64)
    grads = torch.autograd.grad(want, list(h.values()), x["dy"].to(F64))
    assert rel(y, want) <= UNIT[BF] + SUMS
    for got, ref in zip((dx, dw, db), grads):
        assert rel(got, ref) <= 5 * UNIT[BF] + SUMS
    for t, w in ((yw, N), (dxw, K)):
        assert (t[:, :off] == 7).all() and (t[:, off + w:] == 7).all()


def test_only_the_gradients_that_are_wanted():
    x = {n: t.cuda() for n, t in make_linear(70, 64, 96, BF).items()}
    y, saved = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"], activation="silu", save=True)
    full = kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation="silu")
    for i, name in enumerate(("input_grad", "weight_grad", "bias_grad")):
        part = kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation="silu", **{name: False})
        for j in range(3):
            assert part[j] is None if i == j else torch.equal(part[j], full[j])


def test_rows_do_not_meet():
    """NaN in one row of x reaches that row of y alone; in one row of the weight, that column."""
    for M in (9, 200):
        x = {n: t.cuda() for n, t in make_linear(M, 80, 136, BF).items()}
        clean, _ = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"])
        x["x"][4], x["weight"][130] = float("nan"), float("inf")
        y, _ = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"])
        rows, cols = [i for i in range(M) if i != 4], [i for i in range(136) if i != 130]
        assert torch.equal(y[rows][:, cols], clean[rows][:, cols]) and torch.isnan(y[4, cols]).all()


def test_nothing_to_do():
    x = {n: t.cuda() for n, t in make_linear(0, 24, 40, BF).items()}
    y, _ = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"])
    assert y.shape == (0, 40)
    dx, dw, db = kda.kda_linear_bwd(x["dy"], x["x"], x["weight"])
    assert dx.shape == (0, 24) and not dw.any() and not db.any()


def test_the_same_bits_every_time():
    x = {n: t.cuda() for n, t in make_linear(1500, 328, 520, BF).items()}
    first = None
    for _ in range(5):
        y, saved = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"], activation="gelu", save=True)
        out = [y, saved, *kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation="gelu")]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))
