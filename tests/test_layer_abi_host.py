"""The convolution, scan and matrix-product entry points reject bad arguments before touching the GPU
(none of these calls reaches CUDA, except where noted)."""

import ctypes

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from gated_delta_rule_intra_gb300._common import row_stride
from gated_delta_rule_intra_gb300.conv import ConvBwdOpts, ConvFwdOpts, ConvStepOpts
from gated_delta_rule_intra_gb300.linear import LinearBwdOpts, LinearFwdOpts
from gated_delta_rule_intra_gb300.scan import ScanBwdOpts, ScanFwdOpts, ScanStepOpts

(OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_CUDA, ERR_DEVICE, ERR_OVERLAP, ERR_WORKSPACE,
 ERR_OPTION) = range(10)
BASE, SPAN = 1 << 40, 1 << 34  # never-dereferenced device addresses, far apart


def at(i, off=0):
    return BASE + i * SPAN + off


@pytest.fixture(scope="module")
def lib():
    return kda.load_library()


def test_the_ctypes_mirrors_have_the_headers_sizes():
    sizes = {ConvFwdOpts: 48, ConvBwdOpts: 80, ConvStepOpts: 32, ScanFwdOpts: 144, ScanBwdOpts: 168,
             ScanStepOpts: 88, LinearFwdOpts: 80, LinearBwdOpts: 64}
    for mirror, size in sizes.items():
        assert ctypes.sizeof(mirror) == size, mirror


def call(fn, names, ints, opts, given):
    p = {n: at(i) for i, n in enumerate(names)}
    p.update({n: v for n, v in given.items() if n in p})
    return fn(*p.values(), *ints, ctypes.addressof(opts), 0)


def conv_fwd(lib, B=2, T=10, D=8, W=4, dtype=0, wdtype=0, act=1, initial=0, final=0, cu=0, num_seqs=0,
             xs=0, ys=0, **ptr):
    op = ConvFwdOpts(initial_state=initial, final_state=final, cu_seqlens=cu, num_seqs=num_seqs, x_stride=xs,
                     y_stride=ys)
    return call(lib.kda_conv_fwd, ("x", "weight", "bias", "y"), (B, T, D, W, dtype, wdtype, act), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(x=0), ERR_NULL), (dict(weight=0), ERR_NULL), (dict(y=0), ERR_NULL),
    (dict(B=0), ERR_SHAPE), (dict(T=-1), ERR_SHAPE), (dict(D=0), ERR_SHAPE), (dict(W=1), ERR_SHAPE),
    (dict(W=5), ERR_SHAPE), (dict(D=(1 << 28) + 1), ERR_SHAPE), (dict(xs=7), ERR_SHAPE), (dict(ys=-8), ERR_SHAPE),
    (dict(cu=at(9)), ERR_SHAPE), (dict(num_seqs=2), ERR_SHAPE), (dict(B=2, cu=at(9), num_seqs=2), ERR_SHAPE),
    (dict(B=1 << 16, T=1 << 16), ERR_SHAPE),
    (dict(dtype=3), ERR_DTYPE), (dict(wdtype=1), ERR_DTYPE), (dict(dtype=-1, wdtype=-1), ERR_DTYPE),
    (dict(act=2), ERR_OPTION), (dict(act=-1), ERR_OPTION),
    (dict(x=at(0, 1)), ERR_ALIGN), (dict(dtype=2, wdtype=2, y=at(3, 2)), ERR_ALIGN),
    (dict(wdtype=2, weight=at(1, 2)), ERR_ALIGN), (dict(B=1, cu=at(9, 2), num_seqs=1), ERR_ALIGN),
    (dict(y=at(0)), ERR_OVERLAP), (dict(y=at(1)), ERR_OVERLAP),
    (dict(initial=at(8), final=at(8)), ERR_OVERLAP), (dict(final=at(3, 64)), ERR_OVERLAP),
])
def test_conv_fwd_refusals(lib, case, want):
    assert conv_fwd(lib, **case) == want


def conv_bwd(lib, B=2, T=10, D=8, W=4, dtype=0, wdtype=0, act=1, ws=at(12), need=None, dinitial=0, dfinal=0,
             xs=0, dys=0, dxs=0, **ptr):
    if need is None:
        need = lib.kda_conv_bwd_workspace_bytes(B, T, D, W, 0)
    op = ConvBwdOpts(d_initial_state=dinitial, d_final_state=dfinal, workspace=ws, workspace_bytes=need,
                     x_stride=xs, dy_stride=dys, dx_stride=dxs)
    return call(lib.kda_conv_bwd, ("dy", "x", "weight", "bias", "dx", "dweight", "dbias"),
                (B, T, D, W, dtype, wdtype, act), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(dy=0), ERR_NULL), (dict(dx=0), ERR_NULL), (dict(dweight=0), ERR_NULL), (dict(dbias=0), ERR_NULL),
    (dict(W=9), ERR_SHAPE), (dict(dys=3), ERR_SHAPE), (dict(dxs=7), ERR_SHAPE),
    (dict(dtype=5), ERR_DTYPE), (dict(act=3), ERR_OPTION), (dict(dweight=at(5, 2)), ERR_ALIGN),
    (dict(ws=at(12, 8)), ERR_ALIGN), (dict(ws=0), ERR_WORKSPACE), (dict(need=16), ERR_WORKSPACE),
    (dict(dx=at(0)), ERR_OVERLAP), (dict(dx=at(1, 16)), ERR_OVERLAP), (dict(dbias=at(5, 4)), ERR_OVERLAP),
    (dict(dinitial=at(4, 16)), ERR_OVERLAP), (dict(ws=at(0)), ERR_OVERLAP),
])
def test_conv_bwd_refusals(lib, case, want):
    assert conv_bwd(lib, **case) == want


def conv_step(lib, N=3, D=8, W=4, dtype=0, wdtype=0, act=1, indices=0, states=0, xs=0, **ptr):
    op = ConvStepOpts(state_indices=indices, num_states=states, x_stride=xs)
    return call(lib.kda_conv_step, ("x", "weight", "bias", "state", "y"), (N, D, W, dtype, wdtype, act), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(state=0), ERR_NULL), (dict(N=-1), ERR_SHAPE), (dict(N=65536), ERR_SHAPE), (dict(states=2), ERR_SHAPE),
    (dict(states=-1), ERR_SHAPE), (dict(xs=4), ERR_SHAPE), (dict(wdtype=1), ERR_DTYPE),
    (dict(indices=at(9, 1), states=3), ERR_ALIGN), (dict(y=at(3)), ERR_OVERLAP),
    (dict(state=at(0)), ERR_OVERLAP), (dict(indices=at(3), states=3), ERR_OVERLAP),
])
def test_conv_step_refusals(lib, case, want):
    assert conv_step(lib, **case) == want


def scan_fwd(lib, B=2, T=20, D=8, N=16, G=2, dtype=0, z=0, initial=0, final=0, saved=0, saved_bytes=None,
             cu=0, num_seqs=0, ws=at(15), need=None, us=0, Bs=0, ys=0, **ptr):
    if saved_bytes is None:
        saved_bytes = lib.kda_scan_saved_bytes(B, T, D, N, num_seqs)
    if need is None:
        need = lib.kda_scan_fwd_workspace_bytes(B, T, D, N, G, num_seqs)
    op = ScanFwdOpts(z=z, initial_state=initial, final_state=final, saved=saved, saved_bytes=saved_bytes,
                     cu_seqlens=cu, num_seqs=num_seqs, workspace=ws, workspace_bytes=need, u_stride=us,
                     B_stride=Bs, y_stride=ys)
    return call(lib.kda_scan_fwd, ("u", "delta", "A", "B_", "C", "y"), (B, T, D, N, G, dtype), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(u=0), ERR_NULL), (dict(A=0), ERR_NULL), (dict(C=0), ERR_NULL), (dict(y=0), ERR_NULL),
    (dict(B=0), ERR_SHAPE), (dict(T=-2), ERR_SHAPE), (dict(D=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE),
    (dict(N=65), ERR_SHAPE), (dict(D=1 << 23, G=1 << 23, N=64, T=1, B=1), ERR_SHAPE), (dict(G=3), ERR_SHAPE), (dict(G=0), ERR_SHAPE), (dict(us=7), ERR_SHAPE),
    (dict(Bs=31), ERR_SHAPE), (dict(B=2, cu=at(9), num_seqs=1), ERR_SHAPE), (dict(num_seqs=1), ERR_SHAPE),
    (dict(dtype=4, saved_bytes=0), ERR_DTYPE), (dict(u=at(0, 1)), ERR_ALIGN), (dict(A=at(2, 2)), ERR_ALIGN),
    (dict(saved=at(8, 16)), ERR_ALIGN), (dict(dtype=2, z=at(9, 2)), ERR_ALIGN),
    (dict(saved=at(8), saved_bytes=64), ERR_WORKSPACE),
    (dict(T=5000, ws=0), ERR_WORKSPACE), (dict(T=5000, need=8), ERR_WORKSPACE),
    (dict(y=at(0)), ERR_OVERLAP), (dict(y=at(4)), ERR_OVERLAP), (dict(z=at(5)), ERR_OVERLAP),
    (dict(initial=at(9), final=at(9, 64)), ERR_OVERLAP), (dict(saved=at(1)), ERR_OVERLAP),
])
def test_scan_fwd_refusals(lib, case, want):
    assert scan_fwd(lib, **case) == want


def test_scan_buffers(lib):
    """States in front of every eight tokens, two for each started 16, padded to 8, 16, 32 or 64, and a 32-bit
    number a token and channel (rounded up to four); a packed call has a slot more for each sequence."""
    def up(n):
        return -(-n // 256) * 256
    for B, T, D, N, seqs, pad in ((2, 33, 8, 16, 0, 16), (1, 16, 5, 3, 0, 8), (1, 100, 8, 20, 4, 32), (1, 1, 1, 64, 0, 64)):
        slots = T // 16 + seqs if seqs else B * -(-T // 16)
        want = up(2 * slots * D * pad * 4) + up(B * T * -(-D // 4) * 16)
        assert lib.kda_scan_saved_bytes(B, T, D, N, seqs) == want
    assert lib.kda_scan_saved_bytes(1, 16, 8, 65, 0) == 0
    assert lib.kda_scan_fwd_workspace_bytes(8, 4096, 4096, 16, 1, 0) == 0  # channels enough
    assert lib.kda_scan_fwd_workspace_bytes(1, 4096, 64, 16, 1, 0) > 0
    assert lib.kda_scan_fwd_workspace_bytes(1, 4096, 64, 16, 3, 0) == 0  # no such call
    assert lib.kda_scan_bwd_workspace_bytes(1, 64, 64, 16, 1, 0) > 64 * 16 * 2 * 4


def scan_bwd(lib, B=2, T=20, D=8, N=16, G=2, dtype=0, z=0, dz=0, skip=0, dskip=0, bias=0, dbias=0,
             saved=at(14), saved_bytes=None, ws=at(15), need=None, dinitial=0, dfinal=0, dys=0, **ptr):
    if saved_bytes is None:
        saved_bytes = lib.kda_scan_saved_bytes(B, T, D, N, 0)
    if need is None:
        need = lib.kda_scan_bwd_workspace_bytes(B, T, D, N, G, 0)
    op = ScanBwdOpts(z=z, dz=dz, skip=skip, dskip=dskip, delta_bias=bias, ddelta_bias=dbias, saved=saved,
                     saved_bytes=saved_bytes, workspace=ws, workspace_bytes=need, d_initial_state=dinitial,
                     d_final_state=dfinal, dy_stride=dys)
    return call(lib.kda_scan_bwd, ("dy", "u", "delta", "A", "B_", "C", "du", "ddelta", "dA", "dB", "dC"),
                (B, T, D, N, G, dtype), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(dy=0), ERR_NULL), (dict(dA=0), ERR_NULL), (dict(z=at(20)), ERR_NULL), (dict(dz=at(20)), ERR_NULL),
    (dict(skip=at(20)), ERR_NULL), (dict(dbias=at(20)), ERR_NULL), (dict(dys=6), ERR_SHAPE),
    (dict(N=70, need=0, saved_bytes=0), ERR_SHAPE), (dict(dtype=9, saved_bytes=1), ERR_DTYPE),
    (dict(ws=at(15, 128)), ERR_ALIGN), (dict(saved=0), ERR_WORKSPACE), (dict(saved_bytes=256), ERR_WORKSPACE),
    (dict(ws=0), ERR_WORKSPACE), (dict(need=256), ERR_WORKSPACE),
    (dict(du=at(1)), ERR_OVERLAP), (dict(dB=at(10)), ERR_OVERLAP), (dict(ws=at(14)), ERR_OVERLAP),
    (dict(dinitial=at(21), dfinal=at(21)), ERR_OVERLAP),
])
def test_scan_bwd_refusals(lib, case, want):
    assert scan_bwd(lib, **case) == want


def scan_step(lib, R=3, D=8, N=16, G=2, dtype=0, indices=0, states=0, zs=0, z=0, **ptr):
    op = ScanStepOpts(state_indices=indices, num_states=states, z=z, z_stride=zs)
    return call(lib.kda_scan_step, ("u", "delta", "A", "B_", "C", "state", "y"), (R, D, N, G, dtype), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(state=0), ERR_NULL), (dict(A=0), ERR_NULL), (dict(R=-1), ERR_SHAPE), (dict(R=70000), ERR_SHAPE),
    (dict(states=1), ERR_SHAPE), (dict(G=5), ERR_SHAPE), (dict(N=100), ERR_SHAPE), (dict(zs=1), ERR_SHAPE),
    (dict(dtype=7), ERR_DTYPE), (dict(state=at(5, 4)), ERR_ALIGN), (dict(y=at(5)), ERR_OVERLAP),
    (dict(state=at(3)), ERR_OVERLAP), (dict(z=at(6)), ERR_OVERLAP),
])
def test_scan_step_refusals(lib, case, want):
    assert scan_step(lib, **case) == want


def linear_fwd(lib, M=20, K=16, N=24, dtype=0, bias=0, residual=0, saved=0, act=0, xs=0, ws_=0, ys=0, rs=0,
               work=at(12), need=None, **ptr):
    x, w = ptr.get("x", at(0)), ptr.get("weight", at(1))
    if need is None:
        copies = lib.kda_linear_copies(x, xs or K, w, ws_ or K, None, 0)
        need = lib.kda_linear_fwd_workspace_bytes(M, K, N, copies)
    op = LinearFwdOpts(bias=bias, residual=residual, saved=saved, activation=act, x_stride=xs, weight_stride=ws_,
                       y_stride=ys, residual_stride=rs, workspace=work, workspace_bytes=need)
    return call(lib.kda_linear_fwd, ("x", "weight", "y"), (M, K, N, dtype), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(x=0), ERR_NULL), (dict(weight=0), ERR_NULL), (dict(y=0), ERR_NULL),
    (dict(M=-1), ERR_SHAPE), (dict(K=0), ERR_SHAPE), (dict(N=0), ERR_SHAPE), (dict(K=1 << 25), ERR_SHAPE),
    (dict(M=1 << 30, N=1 << 20), ERR_SHAPE), (dict(xs=15), ERR_SHAPE), (dict(ys=23), ERR_SHAPE), (dict(rs=-1), ERR_SHAPE),
    (dict(dtype=2), ERR_DTYPE), (dict(act=4), ERR_OPTION), (dict(act=-1), ERR_OPTION),
    (dict(x=at(0, 1)), ERR_ALIGN), (dict(bias=at(4, 1)), ERR_ALIGN), (dict(work=at(12, 64)), ERR_ALIGN),
    (dict(xs=17, work=0), ERR_WORKSPACE), (dict(M=128, K=8192, N=128, need=256), ERR_WORKSPACE),
    (dict(y=at(0)), ERR_OVERLAP), (dict(y=at(1, 32)), ERR_OVERLAP), (dict(residual=at(2)), ERR_OVERLAP),
    (dict(act=1, saved=at(2, 64)), ERR_OVERLAP),
])
def test_linear_fwd_refusals(lib, case, want):
    assert linear_fwd(lib, **case) == want


def linear_bwd(lib, M=20, K=16, N=24, dtype=0, saved=at(8), act=1, xs=0, dys=0, work=at(12), need=None, **ptr):
    if need is None:
        need = lib.kda_linear_bwd_workspace_bytes(M, K, N, act if 0 <= act <= 3 else 0, 7, 7)
    op = LinearBwdOpts(saved=saved, activation=act, x_stride=xs, dy_stride=dys, workspace=work,
                       workspace_bytes=need)
    return call(lib.kda_linear_bwd, ("dy", "x", "weight", "dx", "dweight", "dbias"), (M, K, N, dtype), op, ptr)


@pytest.mark.parametrize("case,want", [
    (dict(dy=0), ERR_NULL), (dict(x=0), ERR_NULL), (dict(weight=0), ERR_NULL), (dict(saved=0), ERR_NULL),
    (dict(xs=3), ERR_SHAPE), (dict(dys=1), ERR_SHAPE), (dict(N=-4), ERR_SHAPE), (dict(dtype=5), ERR_DTYPE),
    (dict(act=9), ERR_OPTION), (dict(dweight=at(4, 1)), ERR_ALIGN), (dict(work=0), ERR_WORKSPACE),
    (dict(need=64), ERR_WORKSPACE), (dict(dx=at(0)), ERR_OVERLAP), (dict(dbias=at(4)), ERR_OVERLAP),
    (dict(work=at(8)), ERR_OVERLAP),
])
def test_linear_bwd_refusals(lib, case, want):
    assert linear_bwd(lib, **case) == want


def test_copies_are_of_rows_on_no_16_byte_boundary(lib):
    assert lib.kda_linear_copies(at(0), 16, at(1), 24, at(2), 8) == 0
    assert lib.kda_linear_copies(at(0, 2), 16, at(1), 25, at(2), 8) == 3
    assert lib.kda_linear_copies(at(0), 16, at(1), 24, at(2), 12) == 4


def test_good_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("these addresses exist nowhere: only where no device accepts the call")
    for rc in (conv_fwd(lib), conv_bwd(lib), conv_step(lib), scan_fwd(lib), scan_bwd(lib), scan_step(lib),
               linear_fwd(lib), linear_bwd(lib)):
        assert rc in (ERR_DEVICE, ERR_CUDA)


def test_cpu_tensors_and_unknown_activations_are_refused_by_the_binding():
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    v = torch.zeros(1, 4, 1, 16)
    A, h = torch.zeros(8, 16), torch.zeros(4, 8, 16)
    for fn in (lambda: kda.kda_conv_fwd(x, w), lambda: kda.kda_conv_bwd(x, x, w),
               lambda: kda.kda_conv_step(x[0], torch.zeros(4, 3, 8), w),
               lambda: kda.kda_scan_fwd(x, x, A, v, v),
               lambda: kda.kda_scan_bwd(x, x, x, A, v, v, torch.zeros(0, dtype=torch.uint8)),
               lambda: kda.kda_scan_step(x[0], x[0], A, v[0], v[0], h),
               lambda: kda.kda_linear_fwd(x, w.T), lambda: kda.kda_linear_bwd(x, x, w.T)):
        with pytest.raises(ValueError, match="CUDA"):
            fn()
    with pytest.raises(ValueError, match="activation"):
        kda.kda_linear_fwd(x, w.T, activation="tanh")


def test_row_strides():
    """Rows of a slice, of a transposed batch, of one row, of none."""
    x = torch.zeros(3, 5, 20)
    dev = x.get_device()

    def of(t, tail=1):
        return row_stride("t", t, t.shape, t.dtype, dev, tail)

    assert of(x) == 20 and of(x[..., 4:10]) == 20 and of(x[:1, :1, :7]) == 7 and of(x[:, 2]) == 100
    assert of(x[..., 4:16].unflatten(-1, (3, 4)), 2) == 20 and of(x[:0]) == 20 and of(x[:, :0, :6]) == 6
    assert of(x[0, 0, :9]) == 9 and of(x[:1, ::2]) == 40
    for bad in (x.transpose(0, 1), x[..., ::2], x[:, ::2], x.expand(3, 5, 20)[:, :1].expand(3, 4, 20)):
        with pytest.raises(ValueError):
            of(bad)
