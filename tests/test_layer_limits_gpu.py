"""Convolution, scan and matrix product at the ends of their range: sums beyond the 16-bit type, far
tails of a derivative, long memories, and what is left behind when a kernel gives up."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import BF, F32, F64, HF, SCAN, act64, cu, cuda, make_conv, make_linear, rel, tol

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


# ---------------------------------------------------------------------------- long memories
def slow_scan(few, B, T, D, N, seed=3):
    """Sequences whose states last thousands of tokens: (call's inputs, the first `few`'s 64-bit results).
    Only those have a dy, so that all sums over tokens are theirs."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = {"u": torch.randn(B, T, D, device="cuda", generator=g), "z": torch.randn(B, T, D, device="cuda", generator=g),
         "delta": 0.5 * torch.randn(B, T, D, device="cuda", generator=g),
         "B": torch.randn(B, T, 1, N, device="cuda", generator=g),
         "C": torch.randn(B, T, 1, N, device="cuda", generator=g),
         "D": 1 + 0.2 * torch.randn(D, device="cuda", generator=g), "dy": torch.zeros(B, T, D, device="cuda")}
    x["dy"][:few] = torch.randn(few, T, D, device="cuda", generator=g)
    x["A"] = -0.003 * torch.exp(0.3 * torch.randn(D, N, device="cuda", generator=g))
    x["delta_bias"] = torch.linspace(-3.0, -1.5, D, device="cuda")  # step sizes around 0.05 to 0.2
    f = {n: x[n][:few].to(F64) if x[n].shape[0] == B else x[n].to(F64) for n in x}
    s = torch.nn.functional.softplus(f["delta"] + f["delta_bias"])
    h, hs, ys = torch.zeros(few, D, N, dtype=F64, device="cuda"), [], []
    for t in range(T):
        hs.append(h)
        h = torch.exp(s[:, t, :, None] * f["A"]) * h + (s[:, t] * f["u"][:, t])[..., None] * f["B"][:, t]
        ys.append((h * f["C"][:, t]).sum(-1))
    gate = f["z"] * torch.sigmoid(f["z"])
    want = {"y": (torch.stack(ys, 1) + f["D"] * f["u"]) * gate, "state": h}
    dy, carry, dA = f["dy"] * gate, torch.zeros_like(h), torch.zeros_like(f["A"])
    du = torch.empty_like(dy)
    for t in reversed(range(T)):
        a = torch.exp(s[:, t, :, None] * f["A"])
        G = carry + dy[:, t, :, None] * f["C"][:, t]
        du[:, t] = s[:, t] * (G * f["B"][:, t]).sum(-1) + f["D"] * dy[:, t]
        carry = G * a
        dA += (carry * hs[t] * s[:, t, :, None]).sum(0)
    return x, {**want, "du": du, "dA": dA, "d_initial": carry}


def test_states_that_last_thousands_of_tokens():
    """Walked from end to end (as many sequences as fill the card), A around -0.003."""
    few, B, T, D, N = 2, 256, 8192, 64, 16
    x, want = slow_scan(few, B, T, D, N)
    ins, more = [x[n] for n in SCAN[:5]], [x[n] for n in SCAN[5:]]
    assert kda.load_library().kda_scan_fwd_workspace_bytes(B, T, D, N, 1, 0) == 0  # one segment
    y, state, saved = kda.kda_scan_fwd(*ins, *more, save=True, output_final_state=True)
    out = kda.kda_scan_bwd(x["dy"], *ins, saved, *more, output_d_initial_state=True)
    got = {"y": y[:few], "state": state[:few], "du": out[0][:few], "dA": out[2], "d_initial": out[8][:few]}
    # A decay's relative rounding to FP32 below 1 is 2^-25 on the mean of its size (RMS 2^-24 / sqrt 3 with that of
    # the state itself) and of random sign: over the 3000 tokens that a state lasts, sqrt(3000) 4e-8 = 2e-6.
    # What it is off on the mean, a tenth of 2^-25 = 3e-9 a token, is 3000 times that: 9e-6; dA's terms hold a
    # state and its gradient, each of which is off so.
    for name, ref in want.items():
        assert rel(got[name], ref) <= (22e-6 if name == "dA" else 11e-6), name


def test_states_that_last_thousands_of_single_tokens():
    few, B, T, D, N = 2, 2, 8192, 64, 16
    x, want = slow_scan(few, B, T, D, N)
    state = torch.zeros(B, D, N, device="cuda")
    for t in range(T):
        kda.kda_scan_step(x["u"][:, t], x["delta"][:, t], x["A"], x["B"][:, t], x["C"][:, t], state, *(
            x["D"], x["z"][:, t], x["delta_bias"]))
    assert rel(state, want["state"]) <= 11e-6


# ---------------------------------------------------------------------------- derivatives in the tails
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,N", [(1, 16), (40, 15)])
def test_derivatives_in_the_tails(M, N, act):
    """Relative to themselves, where an absolute allowance would let 0 pass."""
    v = torch.tensor([-2.0, -2.5, -3.0, -4.0, -5.0, -6.5, -8.0, -10.0, -13.0, 2.0, 3.0, 5.0, 8.0, 0.5, 0.0, -0.25][:N], dtype=BF)
    x, w = torch.zeros(M, 8, dtype=BF, device="cuda"), torch.zeros(N, 8, dtype=BF, device="cuda")
    saved = kda.kda_linear_fwd(x, w, v.cuda(), activation=act, save=True)[1]
    dy = torch.ones(M, N, dtype=BF, device="cuda")
    got = kda.kda_linear_bwd(dy, x, w, saved, activation=act, input_grad=False, weight_grad=False)[2]
    t = v.to(F64).requires_grad_()
    want = torch.autograd.grad(act64(t, act).sum(), t)[0] * M
    # BF16's rounding of the result, and the exponential's argument (some 120 at -13) rounded to FP32 beside
    # the approximation's 7e-7: 120 2^-24 + 2e-6
    assert ((got.cpu().to(F64) - want).abs() <= want.abs() * (2.0 ** -8 + 1e-5) + 2.0 ** -126).all()


# ---------------------------------------------------------------------------- no tokens
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,W", [(16, 4), (77, 3)])
@pytest.mark.parametrize("packed", [False, True])
def test_a_convolution_of_no_tokens(D, W, packed, dtype):
    """Tensors without elements have no address; the states pass through."""
    x = cuda(make_conv(1 if packed else 2, 0, D, W, dtype, seqs=2))
    p = cu([0, 0]) if packed else None
    for initial in (None, x["initial"]):
        y, last = kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], initial, activation="silu", output_final_state=True,
                                   cu_seqlens=p)
        assert y.shape == x["x"].shape
        assert torch.equal(last, torch.zeros_like(x["initial"]) if initial is None else initial)
        dx, dw, db, di = kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], initial, x["dfinal"],
                                          activation="silu", output_d_initial_state=True, cu_seqlens=p)
        assert dx.shape == y.shape and not dw.any() and not db.any() and torch.equal(di, x["dfinal"])
