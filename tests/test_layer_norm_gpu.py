"""kda_layer_norm_fwd and kda_layer_norm_bwd against the formulas in 64 bits."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda

pytestmark = pytest.mark.gpu

# Outputs are rounded once: the type's unit roundoff, and FP32 sums below it.  Sums over a row
# or a column are trees or runs of up to some thousand terms of random sign: 1e-6.
TOL = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 1e-6}
SUMS = 1e-6


def rel(got, ref):
    got, ref = got.detach().cpu().double(), ref.detach().cpu().double()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    return float((got - ref).norm() / ref.norm().clamp(min=1e-30))


def make(rows, width, dtype, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, width, generator=g) * 2 + offset).to(dtype)
    dy = torch.randn(rows, width, generator=g).to(dtype)
    w = 1 + 0.3 * torch.randn(width, generator=g)
    b = torch.randn(width, generator=g)
    return x, dy, w, b


def reference(x, dy, w, b, eps=1e-5):
    x, dy = x.double(), dy.double()
    w = torch.ones(x.shape[-1]).double() if w is None else w.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    y = xh * w + (0 if b is None else b.double())
    h = dy * w
    dx = rstd * (h - h.mean(-1, keepdim=True) - xh * (h * xh).mean(-1, keepdim=True))
    n = x.shape[-1]
    return (y, mean.flatten(), rstd.flatten(), dx, (dy * xh).reshape(-1, n).sum(0),
            dy.reshape(-1, n).sum(0))


def check(x, dy, w, b, eps=1e-5):
    c = [None if t is None else t.cuda() for t in (x, dy, w, b)]
    y, mean, rstd = kda.kda_layer_norm_fwd(c[0], c[2], c[3], eps)
    dx, dw, db = kda.kda_layer_norm_bwd(c[1], c[0], c[2], mean, rstd)
    ref = reference(x, dy, w, b, eps)
    tol = TOL[x.dtype]
    for name, got, want, t in (("y", y, ref[0], tol + SUMS), ("mean", mean, ref[1], SUMS),
                               ("rstd", rstd, ref[2], SUMS), ("dx", dx, ref[3], tol + SUMS),
                               ("dweight", dw, ref[4], SUMS), ("dbias", db, ref[5], SUMS)):
        assert rel(got, want) <= t, (name, rel(got, want))
    assert y.dtype == dx.dtype == x.dtype and dw.dtype == db.dtype == torch.float32


@pytest.mark.parametrize("dtype", list(TOL))
@pytest.mark.parametrize("width", [8, 40, 100, 128, 129, 256, 257, 500, 512, 1000, 1024, 1111,
                                   2048, 2049, 4096, 5003, 8192, 8193, 16384, 20001])
def test_widths(width, dtype):
    """Every group size, whole and ragged, and rows that one CTA's registers do not hold."""
    x, dy, w, b = make(37, width, dtype, seed=width)
    check(x, dy, w.to(dtype), b.to(dtype))


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 333, 5000])
@pytest.mark.parametrize("width", [128, 300, 2048])
def test_rows(rows, width):
    x, dy, w, b = make(rows, width, torch.bfloat16, seed=rows)
    check(x, dy, w.bfloat16(), b.bfloat16())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_parameters_in_fp32_or_none(dtype):
    x, dy, w, b = make(20, 256, dtype)
    check(x, dy, w, b)
    check(x, dy, w, None)
    check(x, dy, None, None)


def test_leading_dimensions():
    x, dy, w, b = make(24, 128, torch.bfloat16)
    check(x.view(2, 3, 4, 128), dy.view(2, 3, 4, 128), w, b)
    x, dy, w, b = make(1, 128, torch.float32)
    check(x[0], dy[0], w, b)


@pytest.mark.parametrize("dtype", list(TOL))
@pytest.mark.parametrize("width,start,total", [(128, 0, 384), (128, 1, 300), (200, 8, 1000),
                                               (77, 3, 81)])
def test_column_slices(width, start, total, dtype):
    """Rows further apart than they are wide, on and off 16-byte boundaries, in every tensor."""
    rows = 19
    x, dy, w, b = make(rows, total, dtype)
    w, b = w[:width].to(dtype).contiguous(), b[:width].to(dtype).contiguous()
    part = slice(start, start + width)
    xd, dyd = x.cuda()[:, part], dy.cuda()[:, part]
    yb, dxb = (torch.full((rows, total), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    y, mean, rstd = kda.kda_layer_norm_fwd(xd, w.cuda(), b.cuda(), y=yb[:, part])
    dx, dw, db = kda.kda_layer_norm_bwd(dyd, xd, w.cuda(), mean, rstd, dx=dxb[:, part])
    ref = reference(x[:, part], dy[:, part], w, b)
    assert rel(y, ref[0]) <= TOL[dtype] + SUMS and rel(dx, ref[3]) <= TOL[dtype] + SUMS
    assert rel(dw, ref[4]) <= SUMS and rel(db, ref[5]) <= SUMS
    for t in (yb, dxb):  # nothing written beside the slice
        assert (t[:, :start] == 7).all() and (t[:, start + width:] == 7).all()


def test_large_mean():
    """Differences to the mean, not sums of squares: a mean 1000 times the spread."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(50, 1000, generator=g) + 1000
    y, mean, rstd = kda.kda_layer_norm_fwd(x.cuda())
    ref = reference(x, x, None, None)
    # x - mean is exact to the mean's own rounding, 2^-24 * 1000 of a spread of 1
    assert rel(y, ref[0]) <= 1000 * 2.0 ** -23 and rel(rstd, ref[2]) <= 1e-6


def test_constant_rows():
    """No variance: y is the bias, dx follows rstd = eps^-1/2."""
    x = torch.full((4, 256), 3.0)
    _, dy, w, b = make(4, 256, torch.float32)
    check(x, dy, w, b, eps=1e-2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_alone(bad):
    for width in (128, 2048, 9000):
        x, dy, w, b = make(40, width, torch.bfloat16)
        good = kda.kda_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())[0]
        x[7, 3] = bad
        y, mean, rstd = kda.kda_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
        dx = kda.kda_layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean, rstd,
                                    param_grads=False)[0]
        rest = [i for i in range(40) if i != 7]
        assert y[7].isnan().all() and torch.equal(y[rest], good[rest])
        assert torch.isfinite(dx[rest]).all()


def test_gradient_against_differences():
    """Central differences of the 64-bit formula along a direction, step 1e-5."""
    x, dy, w, b = make(9, 300, torch.float32, seed=5)
    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(6), dtype=torch.float64)

    def loss(xx, ww, bb):
        return float((reference(xx, dy, ww, bb)[0] * dy.double()).sum())

    _, mean, rstd = kda.kda_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = kda.kda_layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    h = 1e-5
    for got, diff, at in (
            (dx, loss(x.double() + h * d, w, b) - loss(x.double() - h * d, w, b), d),
            (dw, loss(x, w.double() + h * d[0], b) - loss(x, w.double() - h * d[0], b), d[0]),
            (db, loss(x, w, b.double() + h * d[0]) - loss(x, w, b.double() - h * d[0]), d[0])):
        got = got.double().cpu()
        assert abs(float((got * at).sum()) - diff / (2 * h)) <= 1e-5 * float(got.norm() * at.norm())


def test_the_same_bits_twice():
    x, dy, w, b = (t.cuda() for t in make(3001, 640, torch.bfloat16))
    runs = []
    for _ in range(3):
        y, mean, rstd = kda.kda_layer_norm_fwd(x, w, b)
        runs.append((y, *kda.kda_layer_norm_bwd(dy, x, w, mean, rstd)))
    for r in runs[1:]:
        assert all(torch.equal(a, c) for a, c in zip(runs[0], r))


def test_no_rows():
    x = torch.empty(0, 256, device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(x)
    dx, dw, db = kda.kda_layer_norm_bwd(x, x, None, mean, rstd)
    assert y.shape == dx.shape == (0, 256) and not dw.any() and not db.any()


def test_another_stream():
    x, dy, w, b = (t.cuda() for t in make(4000, 1024, torch.bfloat16))
    y, mean, rstd = kda.kda_layer_norm_fwd(x, w, b)
    want = kda.kda_layer_norm_bwd(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kda.kda_layer_norm_bwd(dy, x, w, mean, rstd, stream=s)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_refusals():
    x, dy, w, b = (t.cuda() for t in make(6, 256, torch.bfloat16))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x.cpu())
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x.double())
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x, w.half())
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x, w[:128])
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x.t())
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x[:1].expand(6, 256))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(x, w, y=x.half())
    with pytest.raises(kda.KdaError):
        kda.kda_layer_norm_fwd(x, w, b, y=x)
    _, mean, rstd = kda.kda_layer_norm_fwd(x)
    with pytest.raises(ValueError):
        kda.kda_layer_norm_bwd(dy[:5], x, None, mean, rstd)
    with pytest.raises(ValueError):
        kda.kda_layer_norm_bwd(dy, x, None, mean[:5], rstd)
    with pytest.raises(kda.KdaError):
        kda.kda_layer_norm_bwd(dy, x, None, mean, rstd, dx=dy)
