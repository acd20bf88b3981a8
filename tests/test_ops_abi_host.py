"""The recurrence, single-token and layer-norm entry points reject bad arguments before touching
the GPU (none of these calls reaches CUDA, except where noted)."""

import ctypes

import pytest

import gated_delta_rule_intra_gb300 as kda
from gated_delta_rule_intra_gb300.recurrence import ChunkBwdOpts, ChunkFwdOpts, StepOpts

(OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_CUDA, ERR_DEVICE, ERR_OVERLAP,
 ERR_WORKSPACE) = range(9)

# Never-dereferenced device addresses, far apart.
BASE, SPAN = 1 << 40, 1 << 34


def at(i, off=0):
    return BASE + i * SPAN + off


@pytest.fixture(scope="module")
def lib():
    return kda.load_library()


def test_the_ctypes_mirrors_have_the_headers_sizes():
    assert ctypes.sizeof(ChunkFwdOpts) == 56
    assert ctypes.sizeof(ChunkBwdOpts) == 72
    assert ctypes.sizeof(StepOpts) == 24


def fwd(lib, B=1, T=64, H=2, dtype=0, HV=0, cu=0, num_seqs=0, initial=0, final=0, saved=0,
        saved_bytes=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "v", "gate", "beta", "o"))}
    p.update(ptr)
    op = ChunkFwdOpts(HV=HV, initial_state=initial, final_state=final, saved=saved,
                      saved_bytes=saved_bytes, cu_seqlens=cu, num_seqs=num_seqs)
    return lib.kda_chunk_fwd(*p.values(), B, T, H, dtype, ctypes.addressof(op), 0)


@pytest.mark.parametrize("case,want", [
    (dict(q=0), ERR_NULL), (dict(gate=0), ERR_NULL), (dict(o=0), ERR_NULL),
    (dict(B=0), ERR_SHAPE), (dict(T=-1), ERR_SHAPE), (dict(H=0), ERR_SHAPE),
    (dict(HV=3), ERR_SHAPE), (dict(HV=-2), ERR_SHAPE),
    (dict(B=2, cu=at(9), num_seqs=3), ERR_SHAPE), (dict(cu=at(9)), ERR_SHAPE),
    (dict(num_seqs=2), ERR_SHAPE), (dict(B=1 << 20, T=1 << 20), ERR_SHAPE),
    (dict(dtype=2), ERR_DTYPE), (dict(dtype=-1), ERR_DTYPE),
    (dict(q=at(0, 8)), ERR_ALIGN), (dict(beta=at(4, 2)), ERR_ALIGN),
    (dict(final=at(10, 4)), ERR_ALIGN), (dict(saved=at(10, 16), saved_bytes=1), ERR_ALIGN),
    (dict(saved=at(10), saved_bytes=1), ERR_WORKSPACE),
    (dict(o=at(2)), ERR_OVERLAP), (dict(o=at(0, 16)), ERR_OVERLAP),
    (dict(initial=at(10), final=at(10, 256)), ERR_OVERLAP),
])
def test_chunk_fwd_refusals(lib, case, want):
    assert fwd(lib, **case) == want


@pytest.mark.parametrize("dtype,state", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_saved_bytes(lib, dtype, state):
    """Per 64-token slot and value head; one slot more per packed sequence."""
    a_slot = 57504 if dtype == 0 and not state else 106496
    for B, T, HV, n in ((1, 64, 1, 0), (3, 65, 4, 0), (1, 1, 2, 0), (1, 200, 2, 5)):
        slots = T // 64 + n + 1 if n else B * -(-T // 64)
        want = -(-slots * HV * a_slot // 256) * 256
        assert lib.kda_chunk_saved_bytes(B, T, HV, n, dtype, state) == want
    assert lib.kda_chunk_saved_bytes(0, 64, 1, 0, dtype, state) == 0
    assert lib.kda_chunk_saved_bytes(2, 64, 1, 3, dtype, state) == 0


def bwd(lib, B=1, T=64, H=2, dtype=0, HV=0, cu=0, num_seqs=0, state=0, saved=at(12),
        workspace=at(13), saved_bytes=None, workspace_bytes=None, dfinal=0, dinitial=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "gate", "beta", "do", "dq", "dk", "dv",
                                         "dgate", "dbeta"))}
    p.update(ptr)
    good = lib.kda_chunk_saved_bytes(B, T, HV or H, num_seqs, dtype, state)
    sb = good if saved_bytes is None else saved_bytes
    wb = lib.kda_chunk_bwd_workspace_bytes(B, T, H, HV or H, num_seqs, dtype, good)
    op = ChunkBwdOpts(HV=HV, d_final_state=dfinal, d_initial_state=dinitial, cu_seqlens=cu,
                      num_seqs=num_seqs, saved=saved, saved_bytes=sb, workspace=workspace,
                      workspace_bytes=wb if workspace_bytes is None else workspace_bytes)
    return lib.kda_chunk_bwd(*p.values(), B, T, H, dtype, ctypes.addressof(op), 0)


@pytest.mark.parametrize("state", [0, 1])
@pytest.mark.parametrize("case,want", [
    (dict(do=0), ERR_NULL), (dict(dbeta=0), ERR_NULL),
    (dict(HV=3), ERR_SHAPE), (dict(B=2, cu=at(14), num_seqs=1), ERR_SHAPE),
    (dict(dtype=3), ERR_DTYPE),
    (dict(do=at(4, 2)), ERR_ALIGN), (dict(dbeta=at(9, 1)), ERR_ALIGN),
    (dict(saved=at(12, 128)), ERR_ALIGN), (dict(workspace=at(13, 64)), ERR_ALIGN),
    (dict(saved=0), ERR_WORKSPACE), (dict(saved_bytes=12345), ERR_WORKSPACE),
    (dict(workspace=0), ERR_WORKSPACE), (dict(workspace_bytes=256), ERR_WORKSPACE),
    (dict(dq=at(6)), ERR_OVERLAP), (dict(dv=at(4, 16)), ERR_OVERLAP),
    (dict(workspace=at(12)), ERR_OVERLAP), (dict(dinitial=at(11), dfinal=at(11)), ERR_OVERLAP),
])
def test_chunk_bwd_refusals(lib, case, want, state):
    assert bwd(lib, state=state, **case) == want


def test_chunk_bwd_needs_options(lib):
    p = [at(i) for i in range(10)]
    assert lib.kda_chunk_bwd(*p, 1, 64, 2, 0, None, 0) == ERR_WORKSPACE


def test_workspace_bytes(lib):
    """A slot's state gradient, Y and scales; grouped value heads add dq and dk of each in FP32."""
    for dtype, state, a_slot in ((0, 0, 49312), (0, 1, 98304), (1, 0, 98304)):
        saved = lib.kda_chunk_saved_bytes(2, 100, 4, 0, dtype, state)
        base = -(-2 * 2 * 4 * a_slot // 256) * 256
        assert lib.kda_chunk_bwd_workspace_bytes(2, 100, 4, 4, 0, dtype, saved) == base
        assert lib.kda_chunk_bwd_workspace_bytes(2, 100, 2, 4, 0, dtype, saved) == (
            base + 2 * 100 * 4 * 128 * 4 * 2)
        assert lib.kda_chunk_bwd_workspace_bytes(2, 100, 4, 4, 0, dtype, saved + 256) == 0


def step(lib, N=2, H=2, dtype=0, HV=0, indices=0, num_states=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("q", "k", "v", "gate", "beta", "state", "o"))}
    p.update(ptr)
    op = StepOpts(HV=HV, state_indices=indices, num_states=num_states)
    return lib.kda_step(*p.values(), N, H, dtype, ctypes.addressof(op), 0)


@pytest.mark.parametrize("case,want", [
    (dict(state=0), ERR_NULL), (dict(v=0), ERR_NULL),
    (dict(N=-1), ERR_SHAPE), (dict(HV=5), ERR_SHAPE), (dict(num_states=1), ERR_SHAPE),
    (dict(num_states=-1), ERR_SHAPE), (dict(dtype=2), ERR_DTYPE),
    (dict(state=at(5, 8)), ERR_ALIGN), (dict(indices=at(8, 2)), ERR_ALIGN),
    (dict(o=at(5, 1024)), ERR_OVERLAP), (dict(o=at(2)), ERR_OVERLAP),
    (dict(indices=at(5), num_states=4), ERR_OVERLAP),
])
def test_step_refusals(lib, case, want):
    assert step(lib, **case) == want


def norm_fwd(lib, rows=4, width=10, dtype=0, wdtype=0, xs=0, ys=0, **ptr):
    p = {n: at(i) for i, n in enumerate(("x", "weight", "bias", "y", "mean", "rstd"))}
    p.update(ptr)
    return lib.kda_layer_norm_fwd(*p.values(), rows, width, 1e-5, dtype, wdtype, xs, ys, 0)


@pytest.mark.parametrize("case,want", [
    (dict(x=0), ERR_NULL), (dict(y=0), ERR_NULL),
    (dict(width=0), ERR_SHAPE), (dict(rows=-1), ERR_SHAPE), (dict(xs=9), ERR_SHAPE),
    (dict(ys=-1), ERR_SHAPE), (dict(rows=1 << 50, width=1 << 10), ERR_SHAPE),
    (dict(dtype=3), ERR_DTYPE), (dict(dtype=0, wdtype=1), ERR_DTYPE),
    (dict(x=at(0, 1)), ERR_ALIGN), (dict(dtype=2, wdtype=2, y=at(3, 2)), ERR_ALIGN),
    (dict(rstd=at(5, 2)), ERR_ALIGN), (dict(wdtype=2, bias=at(2, 2)), ERR_ALIGN),
    (dict(y=at(0, 2)), ERR_OVERLAP), (dict(mean=at(5)), ERR_OVERLAP),
    (dict(y=at(1)), ERR_OVERLAP),
])
def test_layer_norm_fwd_refusals(lib, case, want):
    assert norm_fwd(lib, **case) == want


def norm_bwd(lib, rows=4, width=10, dtype=0, wdtype=0, strides=(0, 0, 0), work=at(9), need=None,
             **ptr):
    p = {n: at(i) for i, n in enumerate(("dy", "x", "weight", "mean", "rstd", "dx", "dweight",
                                         "dbias"))}
    p.update(ptr)
    if need is None:
        need = lib.kda_layer_norm_bwd_workspace_bytes(rows, width)
    return lib.kda_layer_norm_bwd(*p.values(), rows, width, dtype, wdtype, *strides, work, need, 0)


@pytest.mark.parametrize("case,want", [
    (dict(dy=0), ERR_NULL), (dict(mean=0), ERR_NULL), (dict(dweight=0), ERR_NULL),
    (dict(dbias=0), ERR_NULL), (dict(width=-3), ERR_SHAPE), (dict(strides=(9, 0, 0)), ERR_SHAPE),
    (dict(strides=(0, 0, 3)), ERR_SHAPE), (dict(dtype=7), ERR_DTYPE),
    (dict(dx=at(5, 1)), ERR_ALIGN), (dict(work=at(9, 8)), ERR_ALIGN),
    (dict(work=0), ERR_WORKSPACE), (dict(need=16), ERR_WORKSPACE),
    (dict(dx=at(0)), ERR_OVERLAP), (dict(dweight=at(7)), ERR_OVERLAP),
    (dict(work=at(1)), ERR_OVERLAP),
])
def test_layer_norm_bwd_refusals(lib, case, want):
    assert norm_bwd(lib, **case) == want


def test_good_arguments_reach_the_device_check(lib):
    """With everything in order the next thing a call looks at is the device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("these addresses exist nowhere: only where no device accepts the call")
    for rc in (fwd(lib), bwd(lib), bwd(lib, state=1), step(lib), norm_fwd(lib), norm_bwd(lib)):
        assert rc in (ERR_DEVICE, ERR_CUDA)


def test_cpu_tensors_are_refused_by_the_binding():
    import torch
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_chunk_fwd(x, x, x, g, g[..., 0])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_chunk_bwd(x, x, x, g, g[..., 0], x, torch.zeros(0, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_step(x[0], x[0], x[0], g[0], g[0, ..., 0], torch.zeros(4, 2, 128, 128))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_layer_norm_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_layer_norm_bwd(x, x, None, g[..., 0], g[..., 0])
