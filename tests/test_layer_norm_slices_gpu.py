"""Layer norm between column slices of one buffer."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests.test_layer_norm_gpu import SUMS, TOL, make, reference, rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TOL))
@pytest.mark.parametrize("width", [128, 77])
def test_from_one_slice_of_a_buffer_to_another(width, dtype):
    rows = 19
    x, dy, w, b = make(rows, width, dtype, seed=2)
    w, b = w.to(dtype), b.to(dtype)
    buf = torch.full((rows, 4 * width + 3), 7.0, dtype=dtype, device="cuda")
    xs, ys, gs, ds = (buf[:, i * width + (i > 1):(i + 1) * width + (i > 1)] for i in range(4))
    xs.copy_(x)
    gs.copy_(dy)
    y, mean, rstd = kda.kda_layer_norm_fwd(xs, w.cuda(), b.cuda(), y=ys)
    dx, dw, db = kda.kda_layer_norm_bwd(gs, xs, w.cuda(), mean, rstd, dx=ds)
    ref = reference(x, dy, w, b)
    assert rel(ys, ref[0]) <= TOL[dtype] + SUMS and rel(ds, ref[3]) <= TOL[dtype] + SUMS
    assert rel(dw, ref[4]) <= SUMS and rel(db, ref[5]) <= SUMS
    assert torch.equal(xs.cpu(), x) and torch.equal(gs.cpu(), dy)
    assert (buf[:, 2 * width] == 7).all() and (buf[:, 4 * width + 1:] == 7).all()


def test_slices_that_overlap_are_refused():
    buf = torch.zeros(6, 100, device="cuda")
    with pytest.raises(kda.KdaError):
        kda.kda_layer_norm_fwd(buf[:, :50], y=buf[:, 49:99])
    with pytest.raises(kda.KdaError):
        kda.kda_layer_norm_fwd(buf[:, 50:], y=buf[:, :51][:, 1:])
