"""kda_chunk_fwd, kda_chunk_bwd and kda_step against the definition in 64 bits."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._recurrence import (EXTRA, GRADS, NAMES, STATE_TOL, UNIT, cu, cuda, forward64,
                               gradients64, make, rel, states)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def args(x):
    return [x[n] for n in NAMES]


def check_fwd(x, scale=None, S0=None, lens=None, cu_seqlens=None):
    d = cuda(x)
    o, final, saved = kda.kda_chunk_fwd(*args(d), scale=scale,
                                        initial_state=None if S0 is None else S0.cuda(),
                                        output_final_state=True, cu_seqlens=cu_seqlens)
    ro, rf = forward64(x, scale or 128 ** -0.5, S0, lens)
    dt = x["q"].dtype
    assert o.dtype == dt and final.dtype == torch.float32 and saved is None
    if o.numel():
        assert rel(o, ro) <= UNIT[dt] + EXTRA
    assert rel(final, rf) <= STATE_TOL
    return o, final


def run_train(x, do, scale=None, S0=None, dfinal=None, cu_seqlens=None):
    d = cuda(x)
    S0 = None if S0 is None else S0.cuda()
    o, _, saved = kda.kda_chunk_fwd(*args(d), scale=scale, initial_state=S0, save=True,
                                    cu_seqlens=cu_seqlens)
    grads = kda.kda_chunk_bwd(*args(d), do.cuda(), saved, scale=scale,
                              d_final_state=None if dfinal is None else dfinal.cuda(),
                              output_d_initial_state=S0 is not None, cu_seqlens=cu_seqlens)
    return o, grads, saved


def check_bwd(x, seed=5, scale=None, S0=None, dfinal=None, lens=None, cu_seqlens=None):
    dt = x["q"].dtype
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(seed)).to(dt)
    o, grads, _ = run_train(x, do, scale, S0, dfinal, cu_seqlens)
    assert rel(o, forward64(x, scale or 128 ** -0.5, S0, lens)[0]) <= UNIT[dt] + EXTRA
    ref, dS0 = gradients64(x, do, scale or 128 ** -0.5, S0, dfinal, lens)
    for name, g, r in zip(GRADS, grads, ref):
        assert g.dtype == dt, name
        assert rel(g, r) <= UNIT[dt] + EXTRA, (name, rel(g, r))
    if S0 is not None:
        assert rel(grads[5], dS0) <= STATE_TOL
    else:
        assert grads[5] is None
    return grads


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,H,HV,B", [(1, 1, 1, 1), (2, 3, 3, 1), (15, 1, 2, 2), (16, 2, 2, 1),
                                      (17, 1, 1, 3), (64, 1, 1, 1), (65, 2, 6, 1), (130, 1, 1, 2),
                                      (21, 24, 48, 1), (18, 40, 80, 1)])
def test_forward(T, H, HV, B, dtype):
    check_fwd(make(T, H, HV, B, dtype, seed=T), S0=states(B, HV) if T % 2 else None)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,H,HV,B", [(1, 1, 1, 1), (2, 2, 2, 1), (16, 1, 3, 2), (63, 1, 1, 1),
                                      (64, 2, 2, 1), (65, 1, 2, 2), (129, 1, 1, 1),
                                      (20, 40, 80, 1)])
def test_backward(T, H, HV, B, dtype):
    check_bwd(make(T, H, HV, B, dtype, seed=T + 1))


@pytest.mark.parametrize("T", [1, 40, 100])
def test_gradients_through_the_states(T):
    x = make(T, 1, 2, 2, seed=T)
    check_bwd(x, S0=states(2, 2), dfinal=states(2, 2, seed=9), scale=0.3)


def test_a_single_token_has_no_gate_gradient():
    """Nothing precedes the only token: dgate is exactly zero, as in the definition."""
    x = make(1, 2, 2, 3)
    _, grads, _ = run_train(x, x["v"])
    assert not grads[3].any()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens", [[1], [5, 0, 17], [0, 0, 3], [64, 1, 63, 128], [16, 0, 100, 2, 33]])
def test_packed(lens, dtype):
    x = make(sum(lens), 1, 2, 1, dtype, lo=-2.0, seed=len(lens))
    S0 = states(len(lens), 2)
    o, final = check_fwd(x, S0=S0, lens=lens, cu_seqlens=cu(lens))
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(final[i].cpu(), S0[i])
    check_bwd(x, S0=S0, dfinal=states(len(lens), 2, seed=3), lens=lens, cu_seqlens=cu(lens))


def test_tokens_in_no_sequence_are_left_alone():
    """cu_seqlens that covers tokens 3 .. 23 of 40; also one that runs past the end."""
    x = make(40, 1, 2, seed=2)
    d = cuda(x)
    c = cu([12, 8], start=3)
    o = torch.full_like(d["v"], 7.0)
    _, _, saved = kda.kda_chunk_fwd(*args(d), cu_seqlens=c, o=o, save=True)
    assert (o[:, :3] == 7).all() and (o[:, 23:] == 7).all() and (o[:, 3:23] != 7).any()
    outs = {n: torch.full_like(d[m], 7.0).to(BF) for n, m in zip(GRADS, NAMES)}
    kda.kda_chunk_bwd(*args(d), d["v"], saved, cu_seqlens=c, **outs)
    inside = {n: x[n][:, 3:23] for n in NAMES}
    ref, _ = gradients64(inside, x["v"][:, 3:23], lens=[12, 8])
    for n, r in zip(GRADS, ref):
        assert (outs[n][:, :3] == 7).all() and (outs[n][:, 23:] == 7).all()
        assert rel(outs[n][:, 3:23], r) <= UNIT[BF] + EXTRA
    past = torch.tensor([0, 30, 1000], dtype=torch.int32).cuda()
    a = kda.kda_chunk_fwd(*args(d), cu_seqlens=past)[0]
    assert rel(a, forward64(x, lens=[30, 10])[0]) <= UNIT[BF] + EXTRA


@pytest.mark.parametrize("lowest", [float("-inf"), torch.finfo(torch.float32).min, -1e4, -200.0])
def test_gates_that_clear_a_channel(lowest):
    """A decay of zero: equal to the definition with 2^gate = 0, forwards and backwards."""
    x = make(40, 1, 1, seed=4)
    drop = torch.rand(x["gate"].shape, generator=torch.Generator().manual_seed(8)) < 0.2
    drop[:, 20] = True
    low = dict(x, gate=x["gate"].masked_fill(drop, lowest))
    ref = dict(x, gate=x["gate"].masked_fill(drop, -5000.0))
    d = cuda(low)
    o, final, saved = kda.kda_chunk_fwd(*args(d), output_final_state=True, save=True)
    ro, rf = forward64(ref)
    # cumulative gates of 16 tokens reach 16 * 160: their differences carry 2^-12 of a gate
    assert rel(o, ro) <= UNIT[BF] + 1e-3
    assert rel(final, rf) <= 1e-3
    grads = kda.kda_chunk_bwd(*args(d), d["v"], saved)
    want, _ = gradients64(ref, x["v"])
    for name, g, r in zip(GRADS, grads, want):
        assert rel(g, r) <= UNIT[BF] + 1e-3, name


@pytest.mark.parametrize("case", ["gate0", "beta0", "beta1", "q0", "k0", "v0", "do0"])
def test_zeros_and_ones(case):
    x = make(70, 1, 1, seed=6)
    name, value = case[:-1], float(case[-1])
    if name == "do":
        _, grads, _ = run_train(x, torch.zeros_like(x["v"]))
        assert not any(g.any() for g in grads[:5])
        return
    x[name] = torch.full_like(x[name], value)
    check_bwd(x, S0=states(1, 1), dfinal=states(1, 1, seed=2))


def test_nan_stays_where_it_belongs():
    """A NaN in one sequence or head reaches nothing of another."""
    x = make(40, 2, 2, 2, seed=3)
    clean, _, _ = run_train(x, x["v"])
    x["v"][0, 5, 1] = float("nan")
    o, grads, _ = run_train(x, x["v"])
    assert o[0, 5:, 1].isnan().all() and not o[0, :5, 1].isnan().any()
    assert torch.equal(o[1], clean[1]) and torch.equal(o[0, :, 0], clean[0, :, 0])
    for g in grads[:5]:
        assert torch.isfinite(g[1]).all() and torch.isfinite(g[0, :, 0]).all()


def test_large_values_do_not_overflow():
    """States far outside FP16's range: BF16 operands keep FP32's exponents."""
    x = make(40, 1, 1, dtype=BF, seed=3)
    x["v"] = x["v"] * 1e6
    check_bwd(x, S0=states(1, 1) * 1e6)


def test_gradient_against_differences():
    """Central differences of the 64-bit forward along random directions, 1e-4 steps: their
    own error is below 1e-6; the gradients carry their rounding, averaged over a direction."""
    x = make(50, 1, 2, dtype=HF, seed=11)
    gen = torch.Generator().manual_seed(12)
    do = torch.randn(x["v"].shape, generator=gen).to(HF)
    _, grads, _ = run_train(x, do)
    for name, g in zip(NAMES, grads):
        g = g.double().cpu()
        d = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        d = d / d.norm() + g / g.norm()
        at = []
        for sign in (1, -1):
            moved = {n: t.double() for n, t in x.items()}
            moved[name] = moved[name] + sign * 1e-4 * d
            at.append((forward64(moved)[0] * do.double()).sum())
        want = float(at[0] - at[1]) / 2e-4
        assert abs(float((g * d).sum()) - want) <= (UNIT[HF] + EXTRA) * float(g.norm() * d.norm())


def test_the_same_bits_twice_and_from_one_saved():
    x = make(300, 2, 4, 2, seed=1)
    d = cuda(x)
    runs = []
    for _ in range(2):
        o, _, saved = kda.kda_chunk_fwd(*args(d), save=True)
        keep = saved.clone()
        for _ in range(2):
            runs.append((o, *kda.kda_chunk_bwd(*args(d), d["v"], saved)[:5]))
        assert torch.equal(saved, keep)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_training_and_inference_agree():
    """save=True changes nothing about o and the final state."""
    d = cuda(make(100, 2, 2, seed=7))
    a = kda.kda_chunk_fwd(*args(d), output_final_state=True)
    b = kda.kda_chunk_fwd(*args(d), output_final_state=True, save=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("heads", [1, 40, 100])
def test_number_of_heads_does_not_change_a_head(heads):
    """A head's result does not depend on how many run beside it (how dv is split over CTAs)."""
    x = make(40, heads, heads, seed=21)
    d = cuda(x)
    o, grads, _ = run_train(x, x["v"])
    one = {n: t[:, :, :1].contiguous() for n, t in d.items()}
    oo, _, saved = kda.kda_chunk_fwd(*args(one), save=True)
    gg = kda.kda_chunk_bwd(*args(one), one["v"], saved)
    assert torch.equal(oo, o[:, :, :1])
    for a, b in zip(gg[:5], grads[:5]):
        assert torch.equal(a, b[:, :, :1])


def test_no_tokens():
    x = cuda(make(0, 1, 2, 3))
    S0 = states(3, 2).cuda()
    o, final, saved = kda.kda_chunk_fwd(*args(x), initial_state=S0, output_final_state=True,
                                        save=True)
    assert o.shape == (3, 0, 2, 128) and torch.equal(final, S0)
    grads = kda.kda_chunk_bwd(*args(x), x["v"], saved, d_final_state=S0,
                              output_d_initial_state=True)
    assert torch.equal(grads[5], S0) and grads[0].shape == x["q"].shape


def test_another_stream():
    x = make(200, 4, 4, seed=8)
    d = cuda(x)
    want, wg, _ = run_train(x, x["v"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        o, _, saved = kda.kda_chunk_fwd(*args(d), save=True, stream=handle)
        grads = kda.kda_chunk_bwd(*args(d), d["v"], saved, stream=handle)
        s.synchronize()
        assert torch.equal(o, want)
        assert all(torch.equal(a, b) for a, b in zip(grads[:5], wg[:5]))


def test_in_a_graph():
    x = make(100, 2, 2, seed=8)
    d = cuda(x)
    want, wg, _ = run_train(x, x["v"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _, saved = kda.kda_chunk_fwd(*args(d), save=True)
        grads = kda.kda_chunk_bwd(*args(d), d["v"], saved)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and all(torch.equal(a, b) for a, b in zip(grads[:5], wg[:5]))


# ---------------------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N,H,HV", [(1, 1, 1), (3, 2, 4), (1, 16, 16), (5, 20, 80)])
def test_step(N, H, HV, dtype):
    x = make(1, H, HV, N, dtype, lo=-1.0, seed=N)
    S0 = states(N, HV)
    ro, rf = forward64(x, 0.2, S0)
    d = {n: t[:, 0].contiguous() for n, t in cuda(x).items()}
    st = S0.cuda()
    o = kda.kda_step(*args(d), st, scale=0.2)
    assert o.dtype == dtype and rel(o, ro[:, 0]) <= UNIT[dtype]
    assert rel(st, rf) <= 1e-6  # FP32 throughout: sums of 128 products, 2^-24 each


def test_steps_continue_a_prefill():
    """A prompt in one call, then tokens one by one: as the whole sequence at once."""
    x = make(45, 2, 4, 2, seed=13)
    d = cuda(x)
    _, st, _ = kda.kda_chunk_fwd(*[t[:, :40].contiguous() for t in args(d)],
                                 output_final_state=True)
    ro, rf = forward64(x)
    for t in range(40, 45):
        o = kda.kda_step(*[y[:, t].contiguous() for y in args(d)], st)
        assert rel(o, ro[:, t]) <= UNIT[BF] + EXTRA
    assert rel(st, rf) <= STATE_TOL


def test_step_with_state_indices():
    """States named out of order; rows without a request leave every state alone."""
    x = make(1, 1, 2, 4, seed=3)
    pool = states(6, 2)
    idx = [4, -1, 0, 6]
    d = {n: t[:, 0].contiguous() for n, t in cuda(x).items()}
    st = pool.cuda()
    o = kda.kda_step(*args(d), st, state_indices=torch.tensor(idx, dtype=torch.int32).cuda())
    live = [0, 2]
    ro, rf = forward64({n: t[live] for n, t in x.items()}, S0=pool[[4, 0]])
    assert rel(o[live], ro[:, 0]) <= UNIT[BF]
    assert not o[[1, 3]].any()
    assert rel(st[[4, 0]], rf) <= 1e-6
    others = [1, 2, 3, 5]
    assert torch.equal(st[others].cpu(), pool[others])


def test_step_far_into_a_large_pool():
    """State offsets past 2^31 elements (and 2^32 bytes)."""
    HV, n = 64, 2300  # 2300 * 64 * 16384 elements, 9.6 GB
    pool = torch.empty(n, HV, 128, 128, device="cuda")
    S0 = states(1, HV)
    pool[n - 1] = S0[0].cuda()
    x = make(1, HV, HV, 1, seed=3)
    d = {k: t[:, 0].contiguous() for k, t in cuda(x).items()}
    o = kda.kda_step(*args(d), pool,
                     state_indices=torch.tensor([n - 1], dtype=torch.int32).cuda())
    ro, rf = forward64(x, S0=S0)
    assert rel(o, ro[:, 0]) <= UNIT[BF] and rel(pool[n - 1:], rf) <= 1e-6


def test_step_without_requests():
    x = {n: t[:0, 0].contiguous() for n, t in cuda(make(1, 1, 1)).items()}
    assert kda.kda_step(*args(x), torch.empty(0, 1, 128, 128).cuda()).shape == (0, 1, 128)


# ---------------------------------------------------------------------------- refusals
def test_refusals():
    d = cuda(make(20, 2, 4))
    a = args(d)
    bad = [
        ("cpu", [t.cpu() for t in a], {}),
        ("dtype", [a[0].float(), *a[1:]], {}),
        ("k dtype", [a[0], a[1].half(), *a[2:]], {}),
        ("gate dtype", [*a[:3], a[3].half(), a[4]], {}),
        ("beta shape", [*a[:4], a[4][:, :, :2].contiguous()], {}),
        ("heads", [a[0], a[1], *[t[:, :, :3].contiguous() for t in a[2:]]], {}),
        ("width", [a[0][..., :64].contiguous(), a[1][..., :64].contiguous(), *a[2:]], {}),
        ("strided", [a[0].transpose(1, 2).contiguous().transpose(1, 2), *a[1:]], {}),
        ("scale", a, {"scale": 0.0}),
        ("state shape", a, {"initial_state": torch.zeros(2, 4, 128, 128).cuda()}),
        ("cu dtype", a, {"cu_seqlens": torch.tensor([0, 20]).cuda()}),
        ("cu size", a, {"cu_seqlens": torch.tensor([0], dtype=torch.int32).cuda()}),
    ]
    for name, xs, kw in bad:
        with pytest.raises(ValueError):
            kda.kda_chunk_fwd(*xs, **kw)
            pytest.fail(name)
    two = cuda(make(20, 2, 4, 2))
    with pytest.raises(ValueError):
        kda.kda_chunk_fwd(*args(two), cu_seqlens=cu([20]))
    with pytest.raises(kda.KdaError):  # o over v
        kda.kda_chunk_fwd(*a, o=a[2])
    _, _, saved = kda.kda_chunk_fwd(*a, save=True)
    with pytest.raises(ValueError):
        kda.kda_chunk_bwd(*a, d["v"], saved[:-1])
    with pytest.raises(ValueError):
        kda.kda_chunk_bwd(*a, d["v"].float(), saved)
    s = {n: t[:, 0].contiguous() for n, t in d.items()}
    with pytest.raises(ValueError):
        kda.kda_step(*args(s), torch.zeros(1, 4, 128, 128, dtype=BF).cuda())
    with pytest.raises(ValueError):
        kda.kda_step(*args(s), torch.zeros(2, 4, 128, 128).cuda())
    with pytest.raises(ValueError):
        kda.kda_step(*args(s), torch.zeros(1, 4, 128, 128).cuda(),
                     state_indices=torch.zeros(1).cuda())
