"""kda_conv_fwd, kda_conv_bwd and kda_conv_step against the definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import BF, F32, HF, F64, SUMS, conv64, cu, cuda, leaves, make_conv, rel, tol

pytestmark = pytest.mark.gpu


def check(x, act, lens=None, states=False, bias=True, start=0):
    names = ["x", "weight"] + ["bias"] * bias + ["initial"] * states
    h = leaves(x, names)
    want, final = conv64(h["x"], h["weight"], h.get("bias"), h.get("initial"), act, lens, start)
    loss = (want * x["dy"].to(F64)).sum() + ((final * x["dfinal"].to(F64)).sum() if states else 0)
    grads = dict(zip(names, torch.autograd.grad(loss, [h[n] for n in names])))
    c = cuda(x)
    b, i, f = (c[n] if on else None for n, on in (("bias", bias), ("initial", states), ("dfinal", states)))
    packed = None if lens is None else cu(lens, start)
    y, last = kda.kda_conv_fwd(c["x"], c["weight"], b, i, activation=act, output_final_state=states,
                               cu_seqlens=packed)
    dx, dw, db, di = kda.kda_conv_bwd(c["dy"], c["x"], c["weight"], b, i, f, activation=act,
                                      output_d_initial_state=states, cu_seqlens=packed)
    dt = x["x"].dtype
    assert y.dtype == dx.dtype == dt and dw.dtype == db.dtype == F32
    assert rel(y, want) <= tol(dt)
    assert rel(dx, grads["x"]) <= tol(dt)
    assert rel(dw, grads["weight"]) <= SUMS
    if bias:
        assert rel(db, grads["bias"]) <= SUMS
    if states:
        assert torch.equal(last.cpu(), final.detach().to(dt))  # the inputs themselves
        assert rel(di, grads["initial"]) <= tol(dt)
    return y, dx


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T,D", [(1, 8), (2, 256), (3, 33), (7, 264), (8, 1), (9, 100), (64, 128),
                                 (65, 513), (200, 40), (515, 24)])
def test_shapes(T, D, W, dtype):
    check(make_conv(2, T, D, W, dtype, seed=T + D), "silu")


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 66, 130])
def test_states(T, act):
    """Sequences shorter than the state among them, whose last inputs are partly the first ones."""
    for dtype, W in ((BF, 4), (HF, 3), (F32, 2)):
        x = make_conv(3, T, 72, W, dtype, seed=T)
        if T:
            check(x, act, states=True)
            continue
        c = cuda(x)
        y, last = kda.kda_conv_fwd(c["x"], c["weight"], c["bias"], c["initial"], output_final_state=True)
        assert y.shape == c["x"].shape and torch.equal(last, c["initial"])
        dx, dw, db, di = kda.kda_conv_bwd(c["x"], c["x"], c["weight"], c["bias"], c["initial"],
                                          c["dfinal"], output_d_initial_state=True)
        assert torch.equal(di, c["dfinal"]) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("lens,start", [([1, 2, 3, 0, 5, 64, 65, 63, 130], 0), ([20, 0, 45], 11),
                                        ([0, 0, 1], 0), ([300], 0)])
def test_packed(lens, start, dtype):
    T = sum(lens) + (17 if start else 0) + start
    x = make_conv(1, T, 80, 4, dtype, seqs=len(lens), seed=T)
    y, dx = check(x, "silu", lens, states=True, start=start)
    inside = torch.zeros(T, dtype=torch.bool)
    inside[start:start + sum(lens)] = True
    assert not y[0, ~inside].any() and not dx[0, ~inside].any()


def test_packed_outputs_given_keep_what_is_in_no_sequence():
    x = cuda(make_conv(1, 50, 64, 4, seqs=1))
    y, dx = (torch.full((1, 50, 64), 7.0, dtype=BF, device="cuda") for _ in range(2))
    c = cu([30], 5)
    kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], cu_seqlens=c, y=y)
    kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], cu_seqlens=c, dx=dx)
    for t in (y, dx):
        assert (t[0, :5] == 7).all() and (t[0, 35:] == 7).all()


@pytest.mark.parametrize("wdtype", [None, F32])
@pytest.mark.parametrize("start,D,total", [(0, 128, 384), (8, 128, 300), (3, 77, 81)])
def test_column_slices(start, D, total, wdtype):
    x = make_conv(2, 70, total, 4, BF, wdtype, seed=3)
    part = slice(start, start + D)
    s = {**x, "x": x["x"][..., part], "dy": x["dy"][..., part], "weight": x["weight"][part].contiguous(),
         "bias": x["bias"][part].contiguous()}
    h = leaves(s, ("x", "weight", "bias"))
    want, _ = conv64(h["x"], h["weight"], h["bias"], None, "silu")
    grads = torch.autograd.grad((want * s["dy"].to(F64)).sum(), list(h.values()))
    wide = cuda(x)
    yb, dxb = (torch.full((2, 70, total), 7.0, dtype=BF, device="cuda") for _ in range(2))
    w, b = s["weight"].cuda(), s["bias"].cuda()
    kda.kda_conv_fwd(wide["x"][..., part], w, b, activation="silu", y=yb[..., part])
    _, dw, db, _ = kda.kda_conv_bwd(wide["dy"][..., part], wide["x"][..., part], w, b, activation="silu",
                                    dx=dxb[..., part])
    assert rel(yb[..., part], want) <= tol(BF) and rel(dxb[..., part], grads[0]) <= tol(BF)
    assert rel(dw, grads[1]) <= SUMS and rel(db, grads[2]) <= SUMS
    for t in (yb, dxb):
        assert (t[..., :start] == 7).all() and (t[..., start + D:] == 7).all()


def test_no_bias_and_no_parameter_gradients():
    x = make_conv(2, 40, 96, 4)
    check(x, "silu", bias=False)
    c = cuda(x)
    full = kda.kda_conv_bwd(c["dy"], c["x"], c["weight"], c["bias"], activation="silu")
    part = kda.kda_conv_bwd(c["dy"], c["x"], c["weight"], c["bias"], activation="silu", param_grads=False)
    assert torch.equal(full[0], part[0]) and part[1] is None and part[2] is None


def test_neighbouring_sequences_and_channels_do_not_meet():
    """NaN and infinities in one sequence, and in one channel, reach no other."""
    lens = [33, 64, 40]
    x = cuda(make_conv(1, sum(lens), 64, 4, seqs=3))
    c = cu(lens)
    clean = kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], activation="silu", cu_seqlens=c)[0]
    cdx = kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], activation="silu", cu_seqlens=c)[0]
    bad = x["x"].clone()
    bad[0, 33:97] = float("nan")
    bad[0, 50] = float("inf")
    bad[0, :, 7] = float("nan")
    y = kda.kda_conv_fwd(bad, x["weight"], x["bias"], activation="silu", cu_seqlens=c)[0]
    dx = kda.kda_conv_bwd(x["dy"], bad, x["weight"], x["bias"], activation="silu", cu_seqlens=c)[0]
    keep = [i for i in range(64) if i != 7]
    for got, want in ((y, clean), (dx, cdx)):
        assert torch.equal(got[0, :33][:, keep], want[0, :33][:, keep])
        assert torch.equal(got[0, 97:][:, keep], want[0, 97:][:, keep])


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("W,D", [(4, 128), (3, 77), (2, 8), (4, 1030)])
def test_steps_continue_a_prompt(W, D, dtype):
    """A prompt, then token by token: what the whole sequence at once gives, bit for bit in the state."""
    x = cuda(make_conv(3, 9, D, W, dtype, seed=D))
    whole, last = kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], x["initial"], activation="silu",
                                   output_final_state=True)
    _, state = kda.kda_conv_fwd(x["x"][:, :4].contiguous(), x["weight"], x["bias"], x["initial"],
                                activation="silu", output_final_state=True)
    for t in range(4, 9):
        y = kda.kda_conv_step(x["x"][:, t], state, x["weight"], x["bias"], activation="silu")
        assert rel(y, whole[:, t]) <= 2 * tol(dtype)
    assert torch.equal(state, last)


def test_step_with_indices_and_padding_rows():
    x = cuda(make_conv(1, 5, 64, 4))
    states = torch.randn(9, 3, 64, device="cuda").to(BF)
    before = states.clone()
    idx = torch.tensor([4, -1, 0, 9, 7], dtype=torch.int32, device="cuda")
    y = kda.kda_conv_step(x["x"][0], states, x["weight"], x["bias"], activation="silu", state_indices=idx)
    assert not y[1].any() and not y[3].any()
    picked = before[[4, 0, 7]].contiguous()
    want = kda.kda_conv_step(x["x"][0, [0, 2, 4]].contiguous(), picked, x["weight"], x["bias"],
                             activation="silu")
    assert torch.equal(y[[0, 2, 4]], want) and torch.equal(states[[4, 0, 7]], picked)
    rest = [1, 2, 3, 5, 6, 8]
    assert torch.equal(states[rest], before[rest])


def test_malformed_tables_stay_inside():
    """cu_seqlens out of range and out of order: clamped, nothing outside the buffers is touched."""
    x = cuda(make_conv(1, 40, 64, 4, seqs=3))
    for table in ([-5, 10, 1000, 20], [30, 10, 50, 0], [2 ** 31 - 1, -(2 ** 31), 7, 40]):
        c = torch.tensor(table, dtype=torch.int32, device="cuda")
        kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], x["initial"], output_final_state=True, cu_seqlens=c)
        kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["initial"], x["dfinal"],
                         output_d_initial_state=True, cu_seqlens=c)
    torch.cuda.synchronize()


def test_a_large_one_in_pieces():
    """Many CTAs, against the same in pieces (bit for bit: a token's sums do not depend on them)."""
    x = cuda(make_conv(2, 3001, 1024, 4, seed=5))
    y, _ = kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], activation="silu")
    dx, dw, db, _ = kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], activation="silu")
    for b in range(2):
        one = {n: x[n][b:b + 1].contiguous() for n in ("x", "dy")}
        assert torch.equal(kda.kda_conv_fwd(one["x"], x["weight"], x["bias"], activation="silu")[0], y[b:b + 1])
        got = kda.kda_conv_bwd(one["dy"], one["x"], x["weight"], x["bias"], activation="silu")[0]
        assert torch.equal(got, dx[b:b + 1])
    again = kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], activation="silu")
    assert torch.equal(again[1], dw) and torch.equal(again[2], db)
    h = {n: x[n].cpu().double() for n in ("x", "weight", "bias", "dy")}
    pre = torch.nn.functional.pad(h["x"], (0, 0, 3, 0))
    s = sum(pre[:, j:j + 3001] * h["weight"][:, j] for j in range(4)) + h["bias"]
    e = torch.sigmoid(s)
    g = h["dy"] * e * (1 + s * (1 - e))
    want = torch.stack([(g * pre[:, j:j + 3001]).sum((0, 1)) for j in range(4)], 1)
    assert rel(dw, want) <= SUMS and rel(db, g.sum((0, 1))) <= SUMS
