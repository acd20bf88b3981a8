"""dgate and dbeta in FP32: the same sums, not rounded to 16 bits."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._recurrence import EXTRA, NAMES, cu, cuda, gradients64, make, rel, states

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def args(x):
    return [x[n] for n in NAMES]


@pytest.mark.parametrize("dtype,state", [(BF, False), (BF, True), (HF, False)])
@pytest.mark.parametrize("lo", [-0.5, -40.0])
@pytest.mark.parametrize("H,HV,lens", [(2, 2, None), (1, 3, [40, 0, 17, 70]), (1, 8, [65, 3])])
def test_the_sums_before_their_rounding(H, HV, lens, lo, dtype, state):
    T = sum(lens) if lens else 131
    x = make(T, H, HV, dtype=dtype, lo=lo, seed=81)
    c = None if lens is None else cu(lens)
    n = len(lens or [0])
    S0 = states(n, HV) if state else None
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(9)).to(dtype)
    d = cuda(x)
    _, _, saved = kda.kda_chunk_fwd(*args(d), save=True, cu_seqlens=c,
                                    initial_state=None if S0 is None else S0.cuda())
    a = kda.kda_chunk_bwd(*args(d), do.cuda(), saved, cu_seqlens=c)
    b = kda.kda_chunk_bwd(*args(d), do.cuda(), saved, cu_seqlens=c, gate_grads_fp32=True)
    for p, q in zip(a[:3], b[:3]):
        assert torch.equal(p, q)
    want, _ = gradients64(x, do, S0=S0, lens=lens)
    for p, q, r, leaf in zip(a[3:5], b[3:5], want[3:], (x["gate"], x["beta"])):
        assert q.dtype == torch.float32 and q.shape == leaf.shape and torch.equal(q.to(dtype), p)
        # no rounding to hide behind: what the header states beside it
        assert rel(q, r) <= (1e-3 if dtype == BF and not state else EXTRA)


@pytest.mark.parametrize("HV", [3, 8])
def test_tokens_in_no_sequence_and_given_outputs(HV):
    x = cuda(make(60, 1, HV, seed=82))
    c = cu([20, 13], start=5)
    _, _, saved = kda.kda_chunk_fwd(*args(x), cu_seqlens=c, save=True)
    kw = dict(cu_seqlens=c, gate_grads_fp32=True)
    junk = [torch.full((60 * HV * 128,), float("nan"), device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    del junk  # the allocator hands this memory out again
    g = kda.kda_chunk_bwd(*args(x), x["v"], saved, **kw)
    for t in g[:5]:
        assert torch.isfinite(t).all() and not t[:, :5].any() and not t[:, 38:].any()
    mine, beta = torch.full_like(x["gate"], 7.0), torch.full_like(x["beta"], 7.0)
    kda.kda_chunk_bwd(*args(x), x["v"], saved, dgate=mine, dbeta=beta, **kw)
    assert torch.equal(mine[:, 5:38], g[3][:, 5:38]) and torch.equal(beta[:, 5:38], g[4][:, 5:38])
    assert (mine[:, :5] == 7).all() and (beta[:, 38:] == 7).all()
    with pytest.raises(ValueError):
        kda.kda_chunk_bwd(*args(x), x["v"], saved, dgate=torch.empty_like(x["v"]), **kw)
    with pytest.raises(ValueError):
        kda.kda_chunk_bwd(*args(x), x["v"], saved, dgate=mine, cu_seqlens=c)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_through_the_checked_build(dtype):
    x = cuda(make(67, 2, 4, dtype=dtype, seed=83))

    def call():
        _, _, saved = kda.kda_chunk_fwd(*args(x), save=True)
        return kda.kda_chunk_bwd(*args(x), x["v"], saved, gate_grads_fp32=True)[3:5]

    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    with kda.use_library(kda.DEBUG_LIB_PATH):
        kda.kda_debug_set_flags(word)
        try:
            got = call()
            torch.cuda.synchronize()
        finally:
            kda.kda_debug_set_flags(None)
    assert word.item() == 0
    for a, b in zip(got, call()):
        assert rel(a, b) <= 2 * 1e-3
