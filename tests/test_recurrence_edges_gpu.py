"""Where the recurrence kernels leave their usual course: strong gates, inputs out of FP16's
reach, ragged batches; the bounds-checked build; and the binding's two ways in."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from gated_delta_rule_intra_gb300 import norm, recurrence
from tests._recurrence import (EXTRA, GRADS, NAMES, STATE_TOL, UNIT, cu, cuda, forward64,
                               gradients64, make, rel, states)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def args(x):
    return [x[n] for n in NAMES]


def train(x, do, **kw):
    o, _, saved = kda.kda_chunk_fwd(*args(x), save=True, **kw)
    return (o, *kda.kda_chunk_bwd(*args(x), do, saved, **kw)[:5])


def check(x, lens=None, cu_seqlens=None):
    """One rounding to the type and 1e-4, as for every other size."""
    dt = x["q"].dtype
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(9)).to(dt)
    got = train(cuda(x), do.cuda(), cu_seqlens=cu_seqlens)
    ref = (forward64(x, lens=lens)[0], *gradients64(x, do, lens=lens)[0])
    for name, g, r in zip(("o", *GRADS), got, ref):
        assert rel(g, r) <= UNIT[dt] + EXTRA, (name, rel(g, r))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("lo", [-12.0, -40.0, -150.0])
def test_strong_gates(lo, dtype):
    """A channel loses more than 2^-96 inside 16 tokens: the pairs are taken one by one."""
    check(make(70, 1, 2, dtype=dtype, lo=lo, seed=31))


def test_strong_gates_in_a_few_channels():
    x = make(50, 2, 2, seed=32)
    x["gate"][:, :, 1, 5] = -30.0
    check(x)


@pytest.mark.parametrize("what", ["q", "k", "do", "v"])
def test_inputs_out_of_fp16s_reach(what):
    """BF16 training takes FP16 operands where they fit; k is large where beta is small."""
    x = make(40, 2, 2, seed=33)
    f = 2.0 ** 18
    if what in ("q", "v"):
        x[what] = x[what] * f
    if what == "k":
        x["k"], x["beta"] = x["k"] * f, x["beta"] / f ** 2
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(2)).to(BF)
    if what == "do":
        do = do * f
    got = train(cuda(x), do.cuda())
    ref = (forward64(x)[0], *gradients64(x, do)[0])
    for name, g, r in zip(("o", *GRADS), got, ref):
        assert rel(g, r) <= UNIT[BF] + EXTRA, (name, rel(g, r))


def test_one_large_step_among_small_ones():
    """Values that grow and fade by 2^40 from step to step: the state's scale follows."""
    x = make(96, 1, 1, seed=34)
    x["v"][:, 32:48] *= 2.0 ** 40
    x["gate"][:, 48:] -= 8.0
    d = cuda(x)
    o = train(d, d["v"])[0]
    ref = forward64(x)[0]
    for a in range(0, 96, 16):  # each step within a rounding of its own size
        assert rel(o[:, a:a + 16], ref[:, a:a + 16]) <= UNIT[BF] + EXTRA


@pytest.mark.parametrize("dtype", [BF, HF])
def test_more_sequences_than_are_ranked(dtype):
    lens = [(i * 7) % 5 for i in range(140)]
    check(make(sum(lens), 1, 1, dtype=dtype, seed=35), lens, cu(lens))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_one_long_sequence_among_short_ones(dtype):
    lens = [3, 200, 1, 0, 17]
    x = make(sum(lens), 1, 2, dtype=dtype, seed=36)
    check(x, lens, cu(lens))
    S0 = states(5, 2, seed=37)
    o, final, _ = kda.kda_chunk_fwd(*args(cuda(x)), initial_state=S0.cuda(),
                                    output_final_state=True, cu_seqlens=cu(lens))
    ro, rf = forward64(x, S0=S0, lens=lens)
    assert rel(o, ro) <= UNIT[dtype] + EXTRA and rel(final, rf) <= STATE_TOL


@pytest.mark.parametrize("dtype", [BF, HF])
def test_the_order_of_sequences_does_not_matter(dtype):
    """A sequence's results are the same bits wherever it stands in the batch."""
    lens = [40, 7, 130]
    x = make(sum(lens), 2, 2, dtype=dtype, seed=38)
    parts = [{n: t[:, a:a + n_] for n, t in x.items()}
             for a, n_ in zip((0, 40, 47), lens)]
    turned = {n: torch.cat([parts[i][n] for i in (2, 0, 1)], 1) for n in NAMES}
    a = train(cuda(x), x["v"].cuda(), cu_seqlens=cu(lens))
    b = train(cuda(turned), turned["v"].cuda(), cu_seqlens=cu([130, 40, 7]))
    for p, q in zip(a, b):
        assert torch.equal(p[:, :40], q[:, 130:170]) and torch.equal(p[:, 40:47], q[:, 170:])
        assert torch.equal(p[:, 47:], q[:, :130])


def _debug(call):
    """The call through the bounds-checked build: a clean flag word, and both builds within the
    outputs' own tolerance (twice, each being that far from the exact result at most)."""
    ref = call()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    with kda.use_library(kda.DEBUG_LIB_PATH):
        assert kda.kda_debug_checks()
        kda.kda_debug_set_flags(word)
        try:
            got = call()
            torch.cuda.synchronize()
        finally:
            kda.kda_debug_set_flags(None)
    assert word.item() == 0, f"debug checks reported flags {word.item():#x}"
    for a, b in zip(got, ref):
        if a.numel():
            assert rel(a, b) <= 2 * (UNIT.get(a.dtype, STATE_TOL) + EXTRA)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,H,HV,lens", [(1, 1, 1, None), (67, 2, 4, None), (40, 40, 40, None),
                                         (33, 80, 160, None), (122, 2, 2, [5, 0, 64, 53])])
def test_debug_build(T, H, HV, lens, dtype):
    x = cuda(make(T, H, HV, dtype=dtype, seed=T))
    c = None if lens is None else cu(lens)
    n = 1 if lens is None else len(lens)
    S0 = states(n, HV).cuda()
    _debug(lambda: train(x, x["v"], cu_seqlens=c))
    _debug(lambda: kda.kda_chunk_fwd(*args(x), initial_state=S0, output_final_state=True,
                                     cu_seqlens=c)[:2])


def test_debug_build_of_the_step():
    x = cuda(make(0, 2, 4, seed=3, lead=(5,)))
    S = states(7, 4).cuda()
    idx = torch.tensor([6, 0, -1, 3, 9], dtype=torch.int32, device="cuda")
    _debug(lambda: [kda.kda_step(*args(x), S.clone(), state_indices=idx)])


def test_both_ways_into_the_library_agree():
    """The short way and the checked one give the same bits (they make the same call)."""
    x = cuda(make(37, 2, 4, B=2, seed=40))
    S0 = states(2, 4).cuda()
    a = kda.kda_chunk_fwd(*args(x), 0.3, S0, output_final_state=True, save=True)
    b = recurrence._chunk_fwd(*args(x), 0.3, S0, True, True, None, None)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = kda.kda_chunk_fwd(*args(x), save=True)
    ga = kda.kda_chunk_bwd(*args(x), x["v"], a[2])
    gb = recurrence._chunk_bwd(*args(x), x["v"], a[2], None, None, False, None, (None,) * 5)
    assert all(torch.equal(p, q) for p, q in zip(ga[:5], gb[:5])) and ga[5] is gb[5] is None
    y = cuda(make(0, 2, 4, seed=3, lead=(3,)))
    Sa, Sb = states(3, 4).cuda(), states(3, 4).cuda()
    assert torch.equal(kda.kda_step(*args(y), Sa),
                       recurrence._step(*args(y), Sb, None, None, None))
    assert torch.equal(Sa, Sb)
    h = torch.randn(9, 200, device="cuda").to(BF)
    w, bias = torch.randn(200, device="cuda").to(BF), torch.randn(200, device="cuda").to(BF)
    fa = kda.kda_layer_norm_fwd(h, w, bias)
    fb = norm._layer_norm_fwd(h, w, bias, 1e-5, None)
    assert all(torch.equal(p, q) for p, q in zip(fa, fb))
    ga = kda.kda_layer_norm_bwd(h, h, w, *fa[1:])
    gb = norm._layer_norm_bwd(h, h, w, *fa[1:], None, True)
    assert all(torch.equal(p, q) for p, q in zip(ga, gb))


def test_the_short_way_leaves_the_rest_to_the_checks():
    lib = kda.load_library()
    x = cuda(make(8, 2, 2, seed=41))
    a = args(x)
    assert lib.quick_chunk_fwd(*a, None, None, False, False) is not None
    assert lib.quick_chunk_fwd(*a, 0.0, None, False, False) is None  # a scale of 0
    assert lib.quick_chunk_fwd(*a, 1, None, False, False) is None    # not a float
    assert lib.quick_chunk_fwd(*a[:4], x["beta"].to(BF), None, None, False, False) is None
    assert lib.quick_chunk_fwd(a[0].transpose(1, 2), *a[1:], None, None, False, False) is None
    assert lib.quick_chunk_fwd(a[0].cpu(), *a[1:], None, None, False, False) is None
    assert lib.quick_chunk_fwd(a[0], None, *a[2:], None, None, False, False) is None
    saved = torch.empty(17, dtype=torch.uint8, device="cuda")
    assert lib.quick_chunk_bwd(*a, x["v"], saved, None) is None
    h = torch.randn(4, 6, 32, device="cuda")
    assert lib.quick_layer_norm_fwd(h[:, :, :16], None, None, 1e-5) is None  # a slice
    assert lib.quick_layer_norm_fwd(h, None, None, 1e-5) is not None
    o, _, _ = kda.kda_chunk_fwd(*a, 1)  # the checked way takes an integer
    assert torch.equal(o, kda.kda_chunk_fwd(*a, 1.0)[0])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("H,HV", [(1, 3), (2, 2)])
def test_zeros_where_no_sequence_is(H, HV, dtype):
    """Outputs that the call allocates have zeros before the first and behind the last sequence,
    whatever was in their memory."""
    x = cuda(make(50, H, HV, dtype=dtype, seed=42))
    c = cu([20, 0, 13], start=5)
    junk = [torch.full((50 * HV * 128,), float("nan"), device="cuda", dtype=dtype)
            for _ in range(8)]
    torch.cuda.synchronize()
    del junk  # the allocator hands this memory out again
    got = train(x, x["v"], cu_seqlens=c)
    for name, t in zip(("o", *GRADS), got):
        assert (t[:, :5] == 0).all() and (t[:, 38:] == 0).all(), name
        assert torch.isfinite(t).all() and (t[:, 5:38] != 0).any(), name
    mine = torch.full_like(x["q"], 7.0)  # an output that the caller gives keeps what it had
    _, _, saved = kda.kda_chunk_fwd(*args(x), save=True, cu_seqlens=c)
    rest = kda.kda_chunk_bwd(*args(x), x["v"], saved, cu_seqlens=c, dq=mine)
    assert (mine[:, :5] == 7).all() and (mine[:, 38:] == 7).all()
    for name, t in zip(GRADS[1:], rest[1:5]):
        assert (t[:, :5] == 0).all() and (t[:, 38:] == 0).all(), name


@pytest.mark.parametrize("every", [1, 2, 3, 7])
def test_mild_and_other_steps_in_turn(every):
    """BF16 training prepares steps with mild gates and ordinary inputs in a form of their own: the
    forms follow one another, also where a step looks mild and turns out not to be."""
    x = make(16 * 23 + 5, 1, 2, seed=43)
    for step in range(0, 24, every):
        a = slice(16 * step, 16 * step + 16)
        kind = step // every % 4
        if kind == 0:
            x["gate"][:, a, 0, 7] -= 1.9  # a channel loses 2^-30 and more
        elif kind == 1:
            x["k"][:, a] *= 16.0
            x["beta"][:, a] /= 256.0
        elif kind == 2:
            x["q"][:, a] *= 512.0
        else:
            x["gate"][:, a] -= 8.0
    check(x)
