"""Projections, convolution, scan and epilogue run together, as a layer that is trained and served: its
outputs and gradients against the definition in 64 bits, and a prompt read at once, in parts and token
by token."""

import importlib.util
import os

import pytest
import torch

from tests._layer import BF, F64, HF, UNIT, act64, conv64, rel, scan64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# The way through the layer rounds seven times (norm, three projections, convolution, scan, the last
# projection), each by at most a unit of a value that the later ones scale by a few; the way back as
# often.  Sixteen units leave each a gain of two.
ROUNDINGS = 16


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("scan_layer", os.path.join(ROOT, "examples", "scan_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def layer_and_input(example, dtype, T=37, B=2, width=96):
    torch.manual_seed(0)
    layer = example.ScanLayer(width, 136, 8).cuda()
    return layer, torch.randn(B, T, width, device="cuda").to(dtype)


def layer64(layer, p, x):
    """The layer from its definition; p: the parameters in 64 bits, matrices as the layer rounds them."""
    h = torch.nn.functional.layer_norm(x, (x.shape[-1],), p["norm_w"], p["norm_b"])
    v, z = (h @ p["inp"].T).chunk(2, -1)
    u, _ = conv64(v, p["conv_w"], p["conv_b"], None, "silu")
    d, B, C = (u @ p["select"].T).split(layer.sizes, -1)
    y, _ = scan64(u, d @ p["delta"].T, -p["log_A"].exp(), B.unsqueeze(-2), C.unsqueeze(-2), p["skip"], z,
                  p["delta_bias"])
    return x + y @ p["out"].T


@pytest.mark.parametrize("dtype", [BF, HF])
def test_trained(example, dtype):
    layer, x = layer_and_input(example, dtype)
    x.requires_grad_()
    y = layer(x)
    dy = torch.randn_like(y)
    names = [n for n, _ in layer.named_parameters()]
    got = torch.autograd.grad(y, [x, *layer.parameters()], dy)
    p = {}
    for n, t in layer.named_parameters():
        rounded = t.to(dtype) if n in ("inp", "out", "select", "delta") else t
        p[n] = rounded.detach().cpu().to(F64).requires_grad_()
    x64 = x.detach().cpu().to(F64).requires_grad_()
    want = layer64(layer, p, x64)
    ref = torch.autograd.grad(want, [x64, *(p[n] for n in names)], dy.cpu().to(F64))
    limit = ROUNDINGS * UNIT[dtype]
    assert rel(y, want) <= limit
    for n, g, r in zip(("x", *names), got, ref):
        assert rel(g, r) <= limit, (n, rel(g, r))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_served(example, dtype):
    """A prompt and single tokens after it are the sequence read at once (each within the roundings of
    the exact one)."""
    layer, x = layer_and_input(example, dtype, T=29, B=3)
    with torch.no_grad():
        want = layer(x)
    y, states = layer.prefill(x[:, :20].contiguous())
    limit = 2 * ROUNDINGS * UNIT[dtype]
    assert rel(y, want[:, :20]) <= limit
    for t in range(20, 29):
        assert rel(layer.step(x[:, t].contiguous(), states), want[:, t]) <= limit
    _, whole = layer.prefill(x)
    assert rel(states[0], whole[0]) <= limit and rel(states[1], whole[1]) <= limit


def test_the_whole_model_runs(example):
    first, last, right = example.run(3, sequences=4, verbose=False)
    assert all(map(torch.isfinite, map(torch.tensor, (first, last, right))))


def test_a_training_step_in_a_graph(example):
    """Forward and backward captured, after an eager step of the same parameters."""
    layer, x = layer_and_input(example, BF)
    x.requires_grad_()
    leaves = [x, *layer.parameters()]
    dy = torch.randn(x.shape, device="cuda").to(BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = torch.autograd.grad(layer(x), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = torch.autograd.grad(layer(x), leaves, dy)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
