"""Matrix product with bias, activation and residual in its epilogue (``kda_linear_fwd``) and its
gradients (``kda_linear_bwd``).  ``stream=`` (a torch stream or a raw handle) runs a call on another
stream than the current one.

    y = act(x weight^T + bias) + residual
"""

from __future__ import annotations

import ctypes
import math

import torch

from ._common import (ACTIVATIONS, DTYPES16, activation_code, check, library, ptr, row_stride, run,
                      takes_stream)

_GRAD_X, _GRAD_WEIGHT, _GRAD_BIAS = 1, 2, 4  # KDA_GRAD_* of include/kda.h


class LinearFwdOpts(ctypes.Structure):
    """Mirror of kda_linear_fwd_opts_t."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("bias", "residual", "saved")]
                + [("activation", ctypes.c_int)]
                + [(n + "_stride", ctypes.c_longlong) for n in ("x", "weight", "residual", "y")]
                + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)])


class LinearBwdOpts(ctypes.Structure):
    """Mirror of kda_linear_bwd_opts_t."""
    _fields_ = ([("saved", ctypes.c_void_p), ("activation", ctypes.c_int)]
                + [(n + "_stride", ctypes.c_longlong) for n in ("dy", "x", "weight", "dx")]
                + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)])


def _inputs(fn, op, x, weight):
    """Checks of x and weight, whose strides go into `op`; (M, K, N, device index)."""
    dev, dt = x.get_device(), x.dtype
    if dev < 0:
        raise ValueError(f"{fn} needs CUDA tensors (no CPU path exists)")
    if dt not in DTYPES16:
        raise ValueError(f"x must be bf16 or fp16, got {dt}")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x needs a last dimension of at least 1")
    K = x.shape[-1]
    if weight.dim() != 2 or weight.shape[1] != K or weight.shape[0] == 0:
        raise ValueError(f"weight must be [out, {K}], got {tuple(weight.shape)}")
    op.x_stride = row_stride("x", x, x.shape, dt, dev)
    op.weight_stride = row_stride("weight", weight, weight.shape, dt, dev)
    return math.prod(x.shape[:-1]), K, weight.shape[0], dev


def kda_linear_fwd(x, weight, bias=None, residual=None, *, activation=None, save=False, y=None,
                   stream=None):
    """Returns (y, saved).

    x [..., K], weight [N, K], bias [N], residual [..., N], all bf16 or all fp16; rows evenly spaced
    (column slices of wider tensors will do).  ``activation`` None, "silu", "gelu" (x Phi(x)) or
    "relu".  FP32 sums, rounded once behind the residual.  ``saved``, x weight^T + bias in x's dtype, is
    what ``kda_linear_bwd`` needs where there is an activation; None unless ``save``, and without
    one.
    """
    if stream is None and y is None and activation in ACTIVATIONS:
        out = library().quick_linear_fwd(x, weight, bias, residual, ACTIVATIONS[activation], save)
        if out is not None:
            return out
    return _linear_fwd(x, weight, bias, residual, activation, save, y, stream=stream)


@takes_stream
def _linear_fwd(x, weight, bias, residual, activation, save, y):
    op = LinearFwdOpts(activation=activation_code(activation, tuple(ACTIVATIONS)))
    M, K, N, dev = _inputs("kda_linear_fwd", op, x, weight)
    shape, dt = (*x.shape[:-1], N), x.dtype
    if bias is not None:
        check("bias", bias, (N,), dt, dev)
        op.bias = bias.data_ptr()
    if residual is not None:
        op.residual_stride = row_stride("residual", residual, shape, dt, dev)
        op.residual = residual.data_ptr()
    if y is None:
        y = torch.empty(shape, dtype=dt, device=x.device)
    else:
        op.y_stride = row_stride("y", y, shape, dt, dev)
    saved = None
    if save and activation is not None:
        saved = torch.empty(shape, dtype=dt, device=x.device)
        op.saved = saved.data_ptr()
    lib = library()
    copies = lib.kda_linear_copies(x.data_ptr(), op.x_stride, weight.data_ptr(), op.weight_stride, None, 0)
    work = lib.kda_linear_fwd_workspace_bytes(M, K, N, copies)
    ws = torch.empty(work, dtype=torch.uint8, device=x.device)
    op.workspace, op.workspace_bytes = ws.data_ptr(), work
    run("kda_linear_fwd", dev, x.data_ptr(), weight.data_ptr(), y.data_ptr(), M, K, N, DTYPES16[dt],
        ctypes.addressof(op))
    return y, saved


def kda_linear_bwd(dy, x, weight, saved=None, *, activation=None, input_grad=True, weight_grad=True,
                   bias_grad=True, dx=None, stream=None):
    """Gradients of ``kda_linear_fwd``.  Returns (dx, dweight, dbias), all in x's dtype (None where not
    wanted).  x and weight as given to the forward, dy like its y, ``saved`` what it returned with
    ``save=True``.  residual's gradient is dy itself.  Sums are FP32, in a fixed order, and rounded at their
    end.  With an activation what they are made of has 16 bits: the derivative is taken at ``saved``, and dx and
    dweight are products of dpre = dy act'(saved), itself rounded (dbias sums it unrounded).
    """
    if stream is None and dx is None and activation in ACTIVATIONS:
        out = library().quick_linear_bwd(dy, x, weight, saved, ACTIVATIONS[activation], input_grad,
                                         weight_grad, bias_grad)
        if out is not None:
            return out
    return _linear_bwd(dy, x, weight, saved, activation, input_grad, weight_grad, bias_grad, dx,
                       stream=stream)


@takes_stream
def _linear_bwd(dy, x, weight, saved, activation, input_grad, weight_grad, bias_grad, dx):
    op = LinearBwdOpts(activation=activation_code(activation, tuple(ACTIVATIONS)))
    M, K, N, dev = _inputs("kda_linear_bwd", op, x, weight)
    dt = x.dtype
    op.dy_stride = row_stride("dy", dy, (*x.shape[:-1], N), dt, dev)
    if activation is not None:
        if saved is None:
            raise ValueError("saved is needed with an activation: call the forward with save=True")
        check("saved", saved, (*x.shape[:-1], N), dt, dev)
        op.saved = saved.data_ptr()
    if not input_grad:
        dx = None
    elif dx is None:
        dx = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        op.dx_stride = row_stride("dx", dx, x.shape, dt, dev)
    dw = torch.empty((N, K), dtype=dt, device=x.device) if weight_grad else None
    db = torch.empty(N, dtype=dt, device=x.device) if bias_grad else None
    lib = library()
    copies = lib.kda_linear_copies(x.data_ptr(), op.x_stride, weight.data_ptr(), op.weight_stride,
                                   dy.data_ptr(), op.dy_stride)
    wanted = (_GRAD_X * input_grad) | (_GRAD_WEIGHT * weight_grad) | (_GRAD_BIAS * bias_grad)
    work = lib.kda_linear_bwd_workspace_bytes(M, K, N, op.activation, copies, wanted)
    ws = torch.empty(work, dtype=torch.uint8, device=x.device)
    op.workspace, op.workspace_bytes = ws.data_ptr(), work
    run("kda_linear_bwd", dev, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), ptr(dx), ptr(dw), ptr(db),
        M, K, N, DTYPES16[dt], ctypes.addressof(op))
    return dx, dw, db
