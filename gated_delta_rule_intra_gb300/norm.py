"""Layer norm over the last dimension, forward and backward."""

from __future__ import annotations

import torch

from ._common import DTYPES, F32, check, ptr, run, takes_stream


def _rows(name, t, like):
    """(rows, width, stride between rows) of a tensor whose leading dimensions are one run of
    rows; the last dimension is contiguous."""
    if t.device != like.device or t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)} on {like.device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    width = t.shape[-1]
    if t.is_contiguous():
        return width
    stride = t.stride()
    if stride[-1] != 1 and width > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    step = None  # every leading dimension has to continue the one behind it
    for n, s in zip(reversed(t.shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step, run = s, n * s
        elif s == run:
            run = n * s
        else:
            raise ValueError(f"{name}'s rows must be evenly spaced")
    if step is not None and step < width:
        raise ValueError(f"{name}'s rows must not overlap")
    return width if step is None else step


def _params(x, weight, bias):
    wdtype = x.dtype
    for t in (weight, bias):
        if t is not None:
            wdtype = t.dtype
    if wdtype not in (x.dtype, F32):
        raise ValueError(f"weight and bias must be {x.dtype} or float32, got {wdtype}")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            check(name, t, (x.shape[-1],), wdtype, x.device)
    return DTYPES[wdtype]


def _input(fn, x):
    if x.device.type != "cuda":
        raise ValueError(f"{fn} needs CUDA tensors (no CPU path exists)")
    if x.dtype not in DTYPES:
        raise ValueError(f"x must be bf16, fp16 or fp32, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x needs a last dimension of at least 1")


@takes_stream
def kda_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, *, y=None):
    """y = (x - mean) * rstd * weight + bias over the last dimension.  Returns (y, mean, rstd).

    x [..., width] bf16/fp16/fp32; its last dimension is contiguous and its rows are evenly
    spaced (a column slice of a wider tensor will do).  weight and bias [width] in x's dtype or
    fp32 (None: ones, zeros).  y has x's dtype; mean and rstd [rows] are fp32.
    """
    _input("kda_layer_norm_fwd", x)
    wdtype = _params(x, weight, bias)
    xs, width, dev = _rows("x", x, x), x.shape[-1], x.device
    if y is None:
        y, ys = torch.empty(x.shape, dtype=x.dtype, device=dev), width
    else:
        ys = _rows("y", y, x)
    rows = x.numel() // width
    mean, rstd = torch.empty((2, rows), dtype=F32, device=dev).unbind()
    run("kda_layer_norm_fwd", dev, x.data_ptr(), ptr(weight), ptr(bias), y.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), rows, width, eps, DTYPES[x.dtype], wdtype, xs, ys)
    return y, mean, rstd


@takes_stream
def kda_layer_norm_bwd(dy, x, weight, mean, rstd, *, dx=None, param_grads=True):
    """Gradients of ``kda_layer_norm_fwd``.  Returns (dx, dweight, dbias): dx in x's dtype,
    dweight and dbias [width] fp32 summed over the rows in a fixed order (None unless
    ``param_grads``)."""
    from . import load_library
    _input("kda_layer_norm_bwd", x)
    wdtype = _params(x, weight, None)
    xs, dys, width, dev = _rows("x", x, x), _rows("dy", dy, x), x.shape[-1], x.device
    rows = x.numel() // width
    check("mean", mean, (rows,), F32, dev)
    check("rstd", rstd, (rows,), F32, dev)
    if dx is None:
        dx, dxs = torch.empty(x.shape, dtype=x.dtype, device=dev), width
    else:
        dxs = _rows("dx", dx, x)
    dw = db = ws = None
    need = 0
    if param_grads:
        dw, db = torch.empty((2, width), dtype=F32, device=dev).unbind()
        need = load_library().kda_layer_norm_bwd_workspace_bytes(rows, width)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    run("kda_layer_norm_bwd", dev, dy.data_ptr(), x.data_ptr(), ptr(weight), mean.data_ptr(),
        rstd.data_ptr(), dx.data_ptr(), ptr(dw), ptr(db), rows, width, DTYPES[x.dtype], wdtype,
        dys, xs, dxs, ptr(ws), need)
    return dx, dw, db
