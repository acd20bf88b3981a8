"""kda_scan_fwd, kda_scan_bwd and kda_scan_step against the definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import (BF, F32, F64, HF, SCAN, SUMS, cu, cuda, leaves, make_scan, rel, scan64, tol)

pytestmark = pytest.mark.gpu

# dA, dD, ddelta_bias and the states are FP32: products of some thousand factors of 2^-22 and sums of
# them, and decays exp(s A) whose exponent is rounded to 2^-24 of at most some ten.
PARAMS = 1e-5


def check(x, lens=None, states=False, without=(), softplus=True, start=0):
    names = [n for n in SCAN if n not in without] + ["initial"] * states
    h = leaves(x, names)
    args = [h.get(n) for n in SCAN]
    want, final = scan64(*args, h.get("initial"), softplus, lens, start)
    loss = (want * x["dy"].to(F64)).sum() + ((final * x["dfinal"].to(F64)).sum() if states else 0)
    grads = dict(zip(names, torch.autograd.grad(loss, [h[n] for n in names], allow_unused=True)))
    c = cuda(x)
    ins = [c[n] for n in SCAN[:5]]
    more = [None if n in without else c[n] for n in SCAN[5:]]
    packed = None if lens is None else cu(lens, start)
    opts = {"delta_softplus": softplus, "cu_seqlens": packed}
    y, last, saved = kda.kda_scan_fwd(*ins, *more, c["initial"] if states else None, save=True,
                                      output_final_state=states, **opts)
    out = kda.kda_scan_bwd(c["dy"], *ins, saved, *more, c["dfinal"] if states else None,
                           output_d_initial_state=states, **opts)
    dt = x["u"].dtype
    assert rel(y, want) <= tol(dt)
    if states:
        assert rel(last, final) <= PARAMS
        assert rel(out[8], grads["initial"]) <= PARAMS
    for n, got in zip(SCAN, out):
        if n in without:
            assert got is None
            continue
        ref = grads[n] if grads[n] is not None else torch.zeros_like(h[n])
        limit = PARAMS if got.dtype is F32 and n in ("A", "D", "delta_bias") else tol(dt) + PARAMS
        assert rel(got, ref) <= limit, (n, rel(got, ref))
    return y, out


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,D,N,G", [(1, 4, 16, 1), (2, 33, 16, 1), (15, 32, 16, 1), (16, 64, 8, 2),
                                     (17, 130, 4, 1), (33, 8, 32, 2), (40, 12, 64, 1), (31, 40, 7, 4),
                                     (48, 6, 1, 3), (20, 9, 50, 3), (19, 200, 3, 1)])
def test_shapes(T, D, N, G, dtype):
    check(make_scan(2, T, D, N, G, dtype, seed=T + N))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,N", [(1, 16), (17, 16), (40, 5)])
def test_states(T, N, dtype):
    check(make_scan(3, T, 36, N, 1, dtype, seed=T), states=True)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens,start", [([1, 2, 0, 5, 16, 17, 33], 0), ([20, 0, 25], 11), ([0, 1], 0),
                                        ([70], 0)])
def test_packed(lens, start, dtype):
    T = sum(lens) + start + (7 if start else 0)
    x = make_scan(1, T, 40, 16, 2, dtype, seqs=len(lens), seed=T)
    y, out = check(x, lens, states=True, start=start)
    inside = torch.zeros(T, dtype=torch.bool)
    inside[start:start + sum(lens)] = True
    for i, t in ((None, y), (0, out[0]), (1, out[1]), (3, out[3]), (4, out[4]), (6, out[6])):
        assert not t[0, ~inside].any(), i


def test_segments():
    """Few channels and long sequences: cut into segments that are walked side by side."""
    assert kda.load_library().kda_scan_fwd_workspace_bytes(1, 700, 32, 16, 1, 0) > 0
    check(make_scan(1, 700, 32, 16, seed=1), states=True)
    check(make_scan(1, 600, 8, 7, seed=2, dtype=HF), states=True)
    lens = [300, 1, 0, 270, 40]
    check(make_scan(1, sum(lens), 24, 16, 2, seqs=5, seed=3), lens, states=True)


@pytest.mark.parametrize("without", [("z",), ("D",), ("delta_bias",), ("D", "z", "delta_bias")])
def test_optional_inputs(without):
    check(make_scan(2, 21, 24, 16, seed=4), without=without)


def test_step_sizes_as_they_are():
    x = make_scan(2, 30, 24, 16, seed=5)
    x["delta"] = (0.05 + 0.05 * torch.rand(2, 30, 24)).to(BF)
    x["delta_bias"] = 0.1 * torch.rand(24)
    check(x, softplus=False)


def test_zero_step_sizes_keep_the_state():
    """delta far below the softplus's reach (the type's lowest value too), as for padded tokens."""
    x = cuda(make_scan(1, 40, 32, 16, dtype=BF, seed=6))
    for low in (-200.0, torch.finfo(BF).min, float("-inf")):
        delta = x["delta"].clone()
        delta[:, 10:] = low
        args = (x["A"], x["B"], x["C"], x["D"], x["z"], x["delta_bias"], x["initial"])
        _, state, saved = kda.kda_scan_fwd(x["u"], delta, *args, output_final_state=True, save=True)
        cut = [t[:, :10].contiguous() for t in (x["u"], delta, x["B"], x["C"], x["z"])]
        _, want, _ = kda.kda_scan_fwd(cut[0], cut[1], x["A"], cut[2], cut[3], x["D"], cut[4],
                                      x["delta_bias"], x["initial"], output_final_state=True)
        assert torch.equal(state, want)
        out = kda.kda_scan_bwd(x["dy"], x["u"], delta, *args[:3], saved, *args[3:6])
        assert all(torch.isfinite(t).all() for t in out[:8])
        assert not out[1][:, 10:].any()


def test_strong_and_growing_states():
    """Decays to nothing within a token, and states that grow."""
    x = make_scan(1, 40, 16, 16, dtype=F32, seed=7)
    x["A"] = x["A"] * 40
    check(x, states=True)
    x = make_scan(1, 40, 16, 4, dtype=F32, seed=8)
    x["A"] = 0.1 * x["A"].abs()
    check(x, states=True)


def test_channels_and_sequences_do_not_meet():
    """NaN and infinities in one channel or sequence reach no other (but dB and dC, which are sums over
    channels)."""
    lens = [20, 17, 30]
    x = cuda(make_scan(1, 67, 40, 16, seqs=3, seed=9))
    c = cu(lens)

    def call(u):
        y, last, saved = kda.kda_scan_fwd(u, *[x[n] for n in SCAN[1:]], output_final_state=True, save=True,
                                          cu_seqlens=c)
        return y, last, kda.kda_scan_bwd(x["dy"], u, *[x[n] for n in SCAN[1:5]], saved,
                                         *[x[n] for n in SCAN[5:]], cu_seqlens=c)

    bad = x["u"].clone()
    bad[0, 20:37] = float("nan")
    bad[0, 5, 3] = float("inf")
    y, last, out = call(bad)
    y0, last0, out0 = call(x["u"])
    keep = [i for i in range(40) if i != 3]
    rows = list(range(20)) + list(range(37, 67))
    for a, b in ((y, y0), (out[0], out0[0]), (out[1], out0[1]), (out[6], out0[6])):
        assert torch.equal(a[0, rows][:, keep], b[0, rows][:, keep])
    assert torch.equal(last[[0, 2]][:, keep], last0[[0, 2]][:, keep])
    assert torch.equal(out[3][0, 37:], out0[3][0, 37:]) and torch.equal(out[4][0, 37:], out0[4][0, 37:])


@pytest.mark.parametrize("off", [0, 4, 3])
def test_slices_of_wider_tensors(off):
    """u, delta, z, B and C as column slices, on and off the boundaries of four elements."""
    D, N = 36, 16
    x = make_scan(2, 25, D, N, 1, HF, seed=10)
    h = leaves(x, SCAN)
    want, _ = scan64(*[h[n] for n in SCAN])
    grads = dict(zip(SCAN, torch.autograd.grad((want * x["dy"].to(F64)).sum(), list(h.values()))))
    c = cuda(x)

    def wide(t):
        rows = t.flatten(2) if t.dim() == 4 else t
        w = torch.full((2, 25, rows.shape[-1] + off + 5), float("nan"), dtype=HF, device="cuda")
        s = w[..., off:off + rows.shape[-1]]
        s.copy_(rows)
        return s.unflatten(-1, t.shape[2:]) if t.dim() == 4 else s

    for n in ("u", "delta", "z", "B", "C", "dy"):
        c[n] = wide(c[n])
    yw = torch.full((2, 25, D + 9), 7.0, dtype=HF, device="cuda")
    y, _, saved = kda.kda_scan_fwd(*[c[n] for n in SCAN], save=True, y=yw[..., off:off + D])
    assert rel(y, want) <= tol(HF) and (yw[..., off + D:] == 7).all() and (yw[..., :off] == 7).all()
    out = kda.kda_scan_bwd(c["dy"], *[c[n] for n in SCAN[:5]], saved, *[c[n] for n in SCAN[5:]])
    for n, got in zip(SCAN, out):
        assert rel(got, grads[n]) <= (PARAMS if n in ("A", "D", "delta_bias") else tol(HF) + PARAMS), n


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("D,N,G", [(64, 16, 1), (33, 7, 3), (8, 64, 2), (300, 4, 1), (10, 1, 1), (6, 30, 2)])
def test_steps(D, N, G, dtype):
    x = make_scan(7, 1, D, N, G, dtype, seed=D)
    h = leaves(x, SCAN + ("initial",))
    want, final = scan64(*[h[n] for n in SCAN], h["initial"])
    c = cuda(x)
    state = c["initial"].clone()
    ins = [c[n][:, 0] if c[n].dim() > 2 else c[n] for n in SCAN]
    y = kda.kda_scan_step(*ins[:5], state, *ins[5:])
    assert rel(y, want[:, 0]) <= tol(dtype) and rel(state, final) <= PARAMS


@pytest.mark.parametrize("N", [16, 6])
def test_steps_of_many_requests(N):
    """Enough of them that a thread takes four; padding rows and states in any order among them."""
    R, D = 333, 520
    x = make_scan(R, 1, D, N, 2, BF, seed=11)
    c = cuda(x)
    ins = [c[n][:, 0].contiguous() if c[n].dim() > 2 else c[n] for n in SCAN]
    states = torch.randn(400, D, N, device="cuda")
    before = states.clone()
    idx = torch.randperm(400, device="cuda")[:R].to(torch.int32)
    idx[5], idx[200], idx[332] = -1, 400, 2 ** 31 - 1
    y = kda.kda_scan_step(*ins[:5], states, *ins[5:], state_indices=idx)
    live = [i for i in range(R) if i not in (5, 200, 332)]
    assert not y[[5, 200, 332]].any()
    used = idx[live].long()
    x = {n: (t.cpu() if torch.is_tensor(t) else t) for n, t in x.items()}
    h = {n: x[n].double() for n in SCAN}
    want, final = scan64(*[h[n][live] if h[n].dim() > 2 else h[n] for n in SCAN], before[used].cpu().double())
    assert rel(y[live], want[:, 0]) <= tol(BF) and rel(states[used], final) <= PARAMS
    rest = torch.ones(400, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert torch.equal(states[rest], before[rest])


def test_a_prompt_and_steps_are_the_whole_sequence():
    x = cuda(make_scan(2, 24, 64, 16, dtype=F32, seed=12))
    y, last, _ = kda.kda_scan_fwd(*[x[n] for n in SCAN], x["initial"], output_final_state=True)
    cut = [x[n][:, :20].contiguous() if x[n].dim() > 2 else x[n] for n in SCAN]
    _, state, _ = kda.kda_scan_fwd(*cut, x["initial"], output_final_state=True)
    for t in range(20, 24):
        ins = [x[n][:, t] if x[n].dim() > 2 else x[n] for n in SCAN]
        got = kda.kda_scan_step(*ins[:5], state, *ins[5:])
        assert rel(got, y[:, t]) <= SUMS
    assert rel(state, last) <= SUMS


def test_no_tokens():
    x = cuda(make_scan(2, 0, 16, 8))
    y, last, saved = kda.kda_scan_fwd(*[x[n] for n in SCAN], x["initial"], output_final_state=True, save=True)
    assert y.shape == (2, 0, 16) and torch.equal(last, x["initial"])
    out = kda.kda_scan_bwd(x["dy"], *[x[n] for n in SCAN[:5]], saved, *[x[n] for n in SCAN[5:]], x["dfinal"],
                           output_d_initial_state=True)
    assert torch.equal(out[8], x["dfinal"]) and not out[2].any() and not out[5].any() and not out[7].any()


def test_malformed_tables_stay_inside():
    x = cuda(make_scan(1, 40, 16, 16, seqs=3))
    ins, more = [x[n] for n in SCAN[:5]], [x[n] for n in SCAN[5:]]
    for table in ([-5, 10, 1000, 20], [30, 10, 50, 0], [2 ** 31 - 1, -(2 ** 31), 7, 40]):
        c = torch.tensor(table, dtype=torch.int32, device="cuda")
        _, _, saved = kda.kda_scan_fwd(*ins, *more, x["initial"], output_final_state=True, save=True,
                                       cu_seqlens=c)
        kda.kda_scan_bwd(x["dy"], *ins, saved, *more, x["dfinal"], output_d_initial_state=True, cu_seqlens=c)
    torch.cuda.synchronize()


def test_the_same_bits_every_time():
    x = cuda(make_scan(4, 300, 256, 16, 2, seed=13))
    ins, more = [x[n] for n in SCAN[:5]], [x[n] for n in SCAN[5:]]
    first = None
    for _ in range(5):
        y, _, saved = kda.kda_scan_fwd(*ins, *more, save=True)
        out = [y, *kda.kda_scan_bwd(x["dy"], *ins, saved, *more)[:8]]
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(first, out))
