"""Layer norm over the last dimension, forward and backward."""

from __future__ import annotations

import torch

from ._common import DTYPES, F32, check, library, run, takes_stream


def _stride(name, t, like):
    """Elements between the rows of a tensor like `like` whose last dimension is contiguous and
    whose leading dimensions are one evenly spaced run of rows."""
    if t is not like and (t.dtype is not like.dtype or t.shape != like.shape
                          or t.get_device() != like.get_device()):
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


def _input(fn, x, weight, bias):
    """Checks of x and the parameters; (device index, width, rows, the parameters' type)."""
    dev, shape = x.get_device(), x.shape
    if dev < 0:
        raise ValueError(f"{fn} needs CUDA tensors (no CPU path exists)")
    if x.dtype not in DTYPES:
        raise ValueError(f"x must be bf16, fp16 or fp32, got {x.dtype}")
    if not shape or shape[-1] == 0:
        raise ValueError("x needs a last dimension of at least 1")
    width, wdtype = shape[-1], x.dtype
    for t in (weight, bias):
        if t is not None:
            wdtype = t.dtype
    if wdtype is not x.dtype and wdtype is not F32:
        raise ValueError(f"weight and bias must be {x.dtype} or float32, got {wdtype}")
    if weight is not None:
        check("weight", weight, (width,), wdtype, dev)
    if bias is not None:
        check("bias", bias, (width,), wdtype, dev)
    return dev, width, x.numel() // width, DTYPES[wdtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def kda_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, *, y=None, stream=None):
    """y = (x - mean) * rstd * weight + bias over the last dimension.  Returns (y, mean, rstd).

    x [..., width] bf16/fp16/fp32; its last dimension is contiguous and its rows are evenly
    spaced (a column slice of a wider tensor will do).  weight and bias [width] in x's dtype or
    fp32 (None: ones, zeros).  y has x's dtype; mean and rstd [rows] are fp32.
    """
    if stream is None and y is None:
        out = library().quick_layer_norm_fwd(x, weight, bias, eps)
        if out is not None:
            return out
    return _layer_norm_fwd(x, weight, bias, eps, y, stream=stream)


@takes_stream
def _layer_norm_fwd(x, weight, bias, eps, y):
    dev, width, rows, wdtype = _input("kda_layer_norm_fwd", x, weight, bias)
    xs = _stride("x", x, x)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ys = width
    else:
        ys = _stride("y", y, x)
    mean = torch.empty(rows, dtype=F32, device=x.device)
    rstd = torch.empty(rows, dtype=F32, device=x.device)
    run("kda_layer_norm_fwd", dev, x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), rows, width, eps, DTYPES[x.dtype], wdtype, xs, ys)
    return y, mean, rstd


def kda_layer_norm_bwd(dy, x, weight, mean, rstd, *, dx=None, param_grads=True, stream=None):
    """Gradients of ``kda_layer_norm_fwd``.  Returns (dx, dweight, dbias): dx in x's dtype,
    dweight and dbias [width] fp32 summed over the rows in a fixed order (None unless
    ``param_grads``)."""
    if stream is None and dx is None and param_grads:
        out = library().quick_layer_norm_bwd(dy, x, weight, mean, rstd)
        if out is not None:
            return out
    return _layer_norm_bwd(dy, x, weight, mean, rstd, dx, param_grads, stream=stream)


@takes_stream
def _layer_norm_bwd(dy, x, weight, mean, rstd, dx, param_grads):
    dev, width, rows, wdtype = _input("kda_layer_norm_bwd", x, weight, None)
    xs, dys = _stride("x", x, x), _stride("dy", dy, x)
    check("mean", mean, (rows,), F32, dev)
    check("rstd", rstd, (rows,), F32, dev)
    if dx is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dxs = width
    else:
        dxs = _stride("dx", dx, x)
    dw = db = ws = None
    need = 0
    if param_grads:
        dw = torch.empty(width, dtype=F32, device=x.device)
        db = torch.empty(width, dtype=F32, device=x.device)
        need = library().kda_layer_norm_bwd_workspace_bytes(rows, width)
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    run("kda_layer_norm_bwd", dev, dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
        rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), rows, width, DTYPES[x.dtype], wdtype,
        dys, xs, dxs, _ptr(ws), need)
    return dx, dw, db
