"""The example's layer: its training step against the definition in 64 bits, and that a prompt
read at once and one read token by token leave the same outputs and states."""

import importlib.util
import os

import pytest
import torch

from tests._recurrence import EXTRA, UNIT, gradients64, forward64, rel

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("kda_layer",
                                                  os.path.join(ROOT, "examples", "kda_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def layer_and_input(example, T=37, B=2):
    torch.manual_seed(0)
    layer = example.Layer(192, 2, 4).cuda()
    return layer, torch.randn(B, T, 192, device="cuda").to(torch.bfloat16)


def test_the_recurrence_under_autograd(example):
    layer, x = layer_and_input(example)
    names = ("q", "k", "v", "gate", "beta")
    ins = [t.detach().requires_grad_() for t in layer.inputs(x)]
    o = example.Recurrence.apply(*ins)
    do = torch.randn_like(o)
    grads = torch.autograd.grad(o, ins, do)
    host = {n: t.detach().cpu() for n, t in zip(names, ins)}
    want, _ = gradients64(host, do.cpu())
    assert rel(o, forward64(host)[0]) <= UNIT[torch.bfloat16] + EXTRA
    for g, w in zip(grads, want):
        assert rel(g, w) <= UNIT[torch.bfloat16] + EXTRA


def test_layer_norm_under_autograd(example):
    """Against torch's own in 64 bits: one rounding of y and dx; the parameters' gradients are
    FP32 sums of 74 rows of BF16 inputs (2^-24 a term: 1e-5 is ample)."""
    layer, x = layer_and_input(example)
    w = torch.randn(192, device="cuda", requires_grad=True)
    b = torch.randn(192, device="cuda", requires_grad=True)
    x.requires_grad_()
    y = example.LayerNorm.apply(x, w, b)
    dy = torch.randn_like(y)
    got = torch.autograd.grad(y, (x, w, b), dy)
    h = [t.detach().double().requires_grad_() for t in (x, w, b)]
    ref = torch.nn.functional.layer_norm(h[0], (192,), h[1], h[2])
    want = torch.autograd.grad(ref, h, dy.double())
    assert rel(y, ref) <= UNIT[torch.bfloat16]
    assert rel(got[0], want[0]) <= UNIT[torch.bfloat16]
    assert rel(got[1], want[1]) <= 1e-5 and rel(got[2], want[2]) <= 1e-5


def test_prefill_and_steps_agree(example):
    """The state of a prompt read at once and of one read token by token: both within 1e-5 of
    the exact one for the same inputs.  The projections of one row and of many may round
    differently, so the inputs are computed once."""
    layer, x = layer_and_input(example, T=20)
    ins = [t.detach() for t in layer.inputs(x)]
    kda = example.kda
    o, state, _ = kda.kda_chunk_fwd(*ins, output_final_state=True)
    s = torch.zeros_like(state)
    for t in range(20):
        ot = kda.kda_step(*(i[:, t].contiguous() for i in ins), s)
        assert rel(ot, o[:, t]) <= 2 * (UNIT[torch.bfloat16] + EXTRA)
    assert rel(s, state) <= 2e-5
    y, st = layer.prefill(x)
    assert y.shape == x.shape and st.shape == state.shape
    assert layer.step(x[:, 0].contiguous(), st).shape == x[:, 0].shape


def test_it_learns(example):
    """The loss comes down from what a model that knows nothing has (ln 64 = 4.2 at best), and
    decoding from the state repeats the sequences."""
    first, last, right = example.run(verbose=False)
    assert first > 4.0 and last < 0.8 * first and right > 0.9
