"""The recurrence over the whole range of its inputs: scales of either sign, keys and queries of any
size, keys of zero under gates that clear their channel, keys and gates that are not finite, values
near the type's limits under strong gates -- against the definition in 64 bits."""

import ctypes

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from gated_delta_rule_intra_gb300 import recurrence
from tests._recurrence import (EXTRA, F64, GRADS, NAMES, STATE_TOL, cu, cuda, forward64,
                               gradients64, make, rel, states)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# What the header promises beside the rounding of the outputs: 1e-3 for BF16 calls without a
# state, 1e-5 for o and 1e-4 for the gradients otherwise (EXTRA covers both).
TRAIN = 1e-3


def args(x):
    return [x[n] for n in NAMES]


def rounding(ref, dtype):
    """The error of the exact result rounded to `dtype`; 2% for the spread of another sample."""
    ref = ref.detach()
    return 1.02 * float((ref.to(dtype).to(F64) - ref).norm() / ref.norm().clamp(min=1e-30))


def close(name, got, ref, extra):
    bound = rounding(ref, got.dtype) + extra
    assert rel(got, ref) <= bound, (name, rel(got, ref), bound)


def gradient_of(x, seed=9):
    return torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(seed)).to(
        x["v"].dtype)


def check_train(x, scale=None, do=None, lens=None, extra=None, ref=None):
    """Forward and backward without a state; `ref` are the inputs of the definition."""
    dt = x["q"].dtype
    do = gradient_of(x) if do is None else do
    extra = extra or (TRAIN if dt == BF else EXTRA)
    d, c = cuda(x), None if lens is None else cu(lens)
    o, _, saved = kda.kda_chunk_fwd(*args(d), scale=scale, cu_seqlens=c, save=True)
    got = kda.kda_chunk_bwd(*args(d), do.cuda(), saved, scale=scale, cu_seqlens=c)
    s = scale or 128 ** -0.5
    ref = x if ref is None else ref
    close("o", o, forward64(ref, s, None, lens)[0], extra)
    for name, g, r in zip(GRADS, got, gradients64(ref, do, s, None, None, lens)[0]):
        close(name, g, r, extra)


def check_states(x, scale=None, do=None, ref=None, state_tol=STATE_TOL):
    """Forward and backward with the states and their gradients."""
    B, HV = x["v"].shape[0], x["v"].shape[2]
    S0, dS = states(B, HV), states(B, HV, seed=4)
    do = gradient_of(x) if do is None else do
    d = cuda(x)
    o, final, saved = kda.kda_chunk_fwd(*args(d), scale=scale, initial_state=S0.cuda(),
                                        output_final_state=True, save=True)
    got = kda.kda_chunk_bwd(*args(d), do.cuda(), saved, scale=scale, d_final_state=dS.cuda(),
                            output_d_initial_state=True)
    s = scale or 128 ** -0.5
    ref = x if ref is None else ref
    ro, rf = forward64(ref, s, S0)
    close("o", o, ro, EXTRA)
    assert rel(final, rf) <= state_tol, rel(final, rf)
    grads, dS0 = gradients64(ref, do, s, S0, dS)
    for name, g, r in zip(GRADS, got, grads):
        close(name, g, r, EXTRA)
    assert rel(got[5], dS0) <= state_tol, rel(got[5], dS0)


# ------------------------------------------------------------------------ ordinary inputs
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lo", [-0.02, -0.5, -3.0, -8.0])
@pytest.mark.parametrize("T", [40, 131])
def test_errors_beside_the_rounding(T, lo, dtype):
    check_train(make(T, 1, 2, dtype=dtype, lo=lo, seed=51))


# ------------------------------------------------------------------------ scales
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lo", [-0.5, -3.0, -40.0])
@pytest.mark.parametrize("scale", [-128 ** -0.5, -2.0])
def test_negative_scales(scale, lo, dtype):
    check_train(make(100, 1, 2, dtype=dtype, lo=lo, seed=52), scale)


def test_a_negative_scale_in_packed_sequences():
    lens = [70, 1, 0, 33]
    check_train(make(sum(lens), 2, 2, seed=53), -0.25, lens=lens)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_negative_scale_with_states(dtype):
    check_states(make(70, 1, 2, dtype=dtype, seed=54), -0.25)


# ------------------------------------------------------------------------ small inputs
@pytest.mark.parametrize("lo", [-0.5, -3.0, -40.0])
@pytest.mark.parametrize("scale", [1e-3, -1e-6, 1e-9])
def test_small_scales(scale, lo):
    x = make(100, 1, 2, lo=lo, seed=66)
    check_train(x, scale)
    check_states(x, scale)


@pytest.mark.parametrize("lo", [-0.02, -3.0, -40.0])
@pytest.mark.parametrize("power", [-5, -9, -13, -16, -30])
@pytest.mark.parametrize("what", ["k", "q", "qk", "v"])
def test_small_inputs(what, power, lo):
    """BF16 training takes FP16 operands: their power of two follows the inputs."""
    x = make(70, 1, 2, lo=lo, seed=55)
    for n in what:
        x[n] = x[n] * 2.0 ** power
    check_train(x)


@pytest.mark.parametrize("power", [-9, -16, -30])
def test_small_gradients(power):
    x = make(70, 1, 2, seed=56)
    check_train(x, do=gradient_of(x) * 2.0 ** power)


@pytest.mark.parametrize("what", ["k", "q"])
def test_sizes_that_change_from_step_to_step(what):
    """Each step's o is within the bound of its own size."""
    x = make(16 * 7, 1, 2, lo=-0.1, seed=57)
    for step, power in enumerate((0, -12, 3, -25, -7, 5, 0)):
        x[what][:, 16 * step:16 * step + 16] *= 2.0 ** power
    if what == "k":  # the correction of a large key stays a contraction
        x["beta"] = x["beta"] * 2.0 ** -10
    d = cuda(x)
    o = kda.kda_chunk_fwd(*args(d), save=True)[0].cpu()
    ref = forward64(x)[0]
    for a in range(0, 16 * 7, 16):
        close(a, o[:, a:a + 16], ref[:, a:a + 16], TRAIN)


@pytest.mark.parametrize("lo", [-0.5, -40.0])
def test_keys_and_queries_of_zero_in_whole_steps(lo):
    x = make(80, 1, 2, lo=lo, seed=58)
    x["k"][:, 16:32] = 0
    x["q"][:, 48:64] = 0
    check_train(x)


# ------------------------------------------------------------------------ cleared channels
def cleared(x, mask, gate):
    """(inputs with that gate at `mask`, those of the definition, where 2^gate is zero)"""
    return (dict(x, gate=x["gate"].masked_fill(mask, gate)),
            dict(x, gate=x["gate"].masked_fill(mask, -5000.0)))


LOWEST = [float("-inf"), torch.finfo(torch.float32).min, -1e4, -200.0]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gate", LOWEST)
@pytest.mark.parametrize("share", [0.2, 0.75])
def test_cleared_channels(share, gate, dtype):
    """That share of all gates clears its channel, and one token every channel."""
    x = make(40, 1, 2, dtype=dtype, seed=59)
    drop = torch.rand(x["gate"].shape, generator=torch.Generator().manual_seed(8)) < share
    drop[:, 20] = True
    low, ref = cleared(x, drop, gate)
    check_states(low, ref=ref)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("gate", LOWEST)
@pytest.mark.parametrize("share", [0.2, 0.75])
def test_cleared_channels_in_training(share, gate, dtype):
    x = make(40, 1, 2, dtype=dtype, seed=60)
    drop = torch.rand(x["gate"].shape, generator=torch.Generator().manual_seed(8)) < share
    drop[:, 20] = True
    low, ref = cleared(x, drop, gate)
    check_train(low, ref=ref)


def zero_keys(case, dtype):
    x = make(40, 1, 2, dtype=dtype, seed=61)
    drop = torch.zeros(x["gate"].shape, dtype=torch.bool)
    if case == "padding":      # tokens behind the end of a prompt
        drop[:, 25:] = True
        x["k"][:, 25:] = 0
        x["v"][:, 25:] = 0
    elif case == "reset":      # a token that only clears, last in a step of 16
        drop[:, 15] = True
        x["k"][:, 15] = 0
    elif case == "first":      # the same, first in a step
        drop[:, 16] = True
        x["k"][:, 16] = 0
    else:                      # a channel no key uses, forgotten fast
        x["k"][..., 7] = 0
        x["gate"][..., 7] = -10.0
    return cleared(x, drop, float("-inf"))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("case", ["padding", "reset", "first", "channel"])
def test_keys_of_zero_where_a_channel_is_cleared(case, dtype):
    x, ref = zero_keys(case, dtype)
    check_states(x, ref=ref)
    check_train(x, ref=ref)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,at,n", [(16, 0, 12), (16, 0, 10), (32, 18, 11), (40, 5, 12)])
def test_ordinary_gates_behind_a_run_of_cleared_tokens(T, at, n, dtype):
    """Tokens in a row that clear every channel, or lose 2^-100 each, and a few ordinary ones to the
    end of the step."""
    x = make(T, 1, 2, dtype=dtype, lo=-0.3, seed=65)
    drop = torch.zeros(x["gate"].shape, dtype=torch.bool)
    drop[:, at:at + n] = True
    low, ref = cleared(x, drop, float("-inf"))
    check_states(low, ref=ref)
    x["gate"][:, at:at + n] -= 100.0
    check_states(x)


# ------------------------------------------------------------------------ not finite
@pytest.mark.parametrize("dtype,state", [(BF, False), (BF, True), (HF, False)])
@pytest.mark.parametrize("what", ["q", "k", "v", "gate", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_reaches_no_earlier_token(value, what, dtype, state):
    if what == "gate" and value > 0:
        pytest.skip("a gate is not above zero")
    x = make(40, 2, 2, 2, dtype, seed=62)
    ref = forward64(x)[0]
    clean = kda.kda_chunk_fwd(*args(cuda(x)), output_final_state=state)[0]
    x[what][0, 21, 1] = value
    o = kda.kda_chunk_fwd(*args(cuda(x)), output_final_state=state)[0]
    assert torch.equal(o[1], clean[1]) and torch.equal(o[0, :, 0], clean[0, :, 0])
    assert rel(o[0, :21, 1], ref[0, :21, 1]) <= 2.0 ** -8 + EXTRA
    assert not torch.isfinite(o[0, 21, 1]).all()


# ------------------------------------------------------------------------ large values
@pytest.mark.parametrize("power", [20, 40, 60])
def test_large_values_under_strong_gates(power):
    """A channel loses 2^-90 in a step, 2^90 times the values is out of FP32's range."""
    x = make(70, 1, 2, seed=63)
    x["gate"] = -5.6 - 0.05 * x["gate"].abs()
    x["v"] = x["v"] * 2.0 ** power
    check_train(x)
    check_states(x)


# ------------------------------------------------------------------------ heads
@pytest.mark.parametrize("heads", [1, 40, 100, 160])
@pytest.mark.parametrize("dtype,state", [(BF, True), (HF, False), (HF, True)])
def test_number_of_heads_does_not_change_a_head(heads, dtype, state):
    """Heads run in one, two or four CTAs, by how many there are: the same bits."""
    x = cuda(make(40, heads, heads, dtype=dtype, seed=64))
    S0 = states(1, heads).cuda() if state else None
    dS = states(1, heads, seed=4).cuda() if state else None

    def run(x, S0, dS):
        o, final, saved = kda.kda_chunk_fwd(*args(x), initial_state=S0, save=True,
                                            output_final_state=state)
        return (o, *kda.kda_chunk_bwd(*args(x), x["v"], saved, d_final_state=dS,
                                      output_d_initial_state=state), final)

    many = run(x, S0, dS)
    one = run({n: t[:, :, :1].contiguous() for n, t in x.items()},
              *(t if t is None else t[:, :1].contiguous() for t in (S0, dS)))
    for a, b in zip(one[:6], many[:6]):
        assert torch.equal(a, b[:, :, :1])
    if state:
        for a, b in zip(one[6:], many[6:]):
            assert torch.equal(a, b[:, :1])


# ------------------------------------------------------------------------ zeros
@pytest.mark.parametrize("HV", [8, 3])
def test_zeros_in_a_dbeta_on_any_two_byte_boundary(HV):
    """The C entry takes dbeta on a 2-byte boundary; rows of 8 heads are 16 bytes long."""
    x = cuda(make(50, 1, HV, seed=67))
    c = cu([20, 13], start=5)
    _, _, saved = kda.kda_chunk_fwd(*args(x), cu_seqlens=c, save=True)
    want = kda.kda_chunk_bwd(*args(x), x["v"], saved, cu_seqlens=c)[:5]
    q, k, v, gate, beta = args(x)
    out = [torch.full_like(t, 7.0) for t in want]
    room = torch.full((50 * HV + 3,), 7.0, dtype=BF, device="cuda")
    dbeta = room[1:-2]
    assert dbeta.data_ptr() % 16 == 2
    lib = kda.load_library()
    size = lib.kda_chunk_bwd_workspace_bytes(1, 50, 1, HV, 2, 0, saved.numel())
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    op = recurrence.ChunkBwdOpts(HV=HV, cu_seqlens=c.data_ptr(), num_seqs=2, zero_rest=1,
                                 saved=saved.data_ptr(), saved_bytes=saved.numel(),
                                 workspace=work.data_ptr(), workspace_bytes=size)
    rc = lib.kda_chunk_bwd(q.data_ptr(), k.data_ptr(), gate.data_ptr(), beta.data_ptr(),
                           v.data_ptr(), *[t.data_ptr() for t in out[:4]], dbeta.data_ptr(), 1, 50,
                           1, 0, ctypes.addressof(op), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    for a, b in zip((*out[:4], dbeta.view_as(want[4])), want):
        assert torch.equal(a, b)
    assert room[0] == 7 and (room[-2:] == 7).all()


# ------------------------------------------------------------------------ the caller's choice
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lens", [None, [40, 0, 61]])
def test_precise_calls_without_a_state(lens, dtype):
    """``precise``: the kernels of the calls with a state, the same bits forwards and backwards."""
    x = cuda(make(101, 1, 2, dtype=dtype, seed=68))
    c = None if lens is None else cu(lens)
    do = gradient_of(x).cuda()
    want, _, saved = kda.kda_chunk_fwd(*args(x), cu_seqlens=c, save=True, output_final_state=True)
    grads = kda.kda_chunk_bwd(*args(x), do, saved, cu_seqlens=c)[:5]
    o, final, mine = kda.kda_chunk_fwd(*args(x), cu_seqlens=c, save=True, precise=True)
    assert final is None and mine.numel() == saved.numel() and torch.equal(o, want)
    for a, b in zip(kda.kda_chunk_bwd(*args(x), do, mine, cu_seqlens=c)[:5], grads):
        assert torch.equal(a, b)
    o, final, mine = kda.kda_chunk_fwd(*args(x), cu_seqlens=c, precise=True)
    assert final is None and mine is None and torch.equal(o, want)
    ref = {n: t.cpu() for n, t in x.items()}
    close("o", o, forward64(ref, lens=lens)[0], 1e-5)
    for name, g, r in zip(GRADS, grads, gradients64(ref, do.cpu(), lens=lens)[0]):
        close(name, g, r, EXTRA)


@pytest.mark.parametrize("what", ["v", "do"])
@pytest.mark.parametrize("power", [-60, 60, 90])
@pytest.mark.parametrize("lo", [-0.5, -3.0, -40.0])
def test_values_and_gradients_of_any_size(lo, power, what):
    """As far as the header goes: 2^-80 to 2^100, a little room for sums left."""
    x = make(70, 1, 2, lo=lo, seed=69)
    do = gradient_of(x)
    if what == "v":
        x["v"] = x["v"] * 2.0 ** power
    else:
        do = do * 2.0 ** power
    check_train(x, do=do)


@pytest.mark.parametrize("lo", [-0.1, -3.0])
def test_channels_that_no_key_or_query_uses(lo):
    x = make(70, 1, 2, lo=lo, seed=70)
    x["k"][..., 64:] = 0
    x["q"][..., :32] = 0
    check_train(x)
