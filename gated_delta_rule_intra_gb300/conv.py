"""The short causal convolution of each channel (in front of q, k and v, or of the scan), over whole
sequences and for single tokens.  ``stream=`` (a torch stream or a raw handle) runs a call on another
stream than the current one.

    pre[t, d] = bias[d] + sum_j weight[d, j] x[t - W + 1 + j, d],  y = act(pre)
"""

from __future__ import annotations

import ctypes

import torch

from ._common import (DTYPES, F32, activation_code, check, library, ptr, row_stride, run, sequences,
                      takes_stream)

_ALLOWED = (None, "silu")


class ConvFwdOpts(ctypes.Structure):
    """Mirror of kda_conv_fwd_opts_t."""
    _fields_ = [("initial_state", ctypes.c_void_p), ("final_state", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("zero_rest", ctypes.c_int), ("x_stride", ctypes.c_longlong),
                ("y_stride", ctypes.c_longlong)]


class ConvBwdOpts(ctypes.Structure):
    """Mirror of kda_conv_bwd_opts_t."""
    _fields_ = [("initial_state", ctypes.c_void_p), ("d_final_state", ctypes.c_void_p),
                ("d_initial_state", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("num_seqs", ctypes.c_int), ("zero_rest", ctypes.c_int),
                ("dy_stride", ctypes.c_longlong), ("x_stride", ctypes.c_longlong),
                ("dx_stride", ctypes.c_longlong), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class ConvStepOpts(ctypes.Structure):
    """Mirror of kda_conv_step_opts_t."""
    _fields_ = [("state_indices", ctypes.c_void_p), ("num_states", ctypes.c_int),
                ("x_stride", ctypes.c_longlong), ("y_stride", ctypes.c_longlong)]


def _inputs(fn, x, weight, bias, lead):
    """Checks of x and the parameters; (D, W, device index, the parameters' type)."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{fn} needs CUDA tensors (no CPU path exists)")
    if x.dtype not in DTYPES:
        raise ValueError(f"x must be bf16, fp16 or fp32, got {x.dtype}")
    if x.dim() != lead + 1 or x.shape[-1] == 0:
        raise ValueError(f"x must be [{'N' if lead == 1 else 'B, T'}, D], got {tuple(x.shape)}")
    D = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != D or not 2 <= weight.shape[1] <= 4:
        raise ValueError(f"weight must be [{D}, W] with W 2 to 4, got {tuple(weight.shape)}")
    if weight.dtype is not x.dtype and weight.dtype is not F32:
        raise ValueError(f"weight and bias must be {x.dtype} or float32, got {weight.dtype}")
    check("weight", weight, weight.shape, weight.dtype, dev)
    if bias is not None:
        check("bias", bias, (D,), weight.dtype, dev)
    return D, weight.shape[1], dev, DTYPES[weight.dtype]


def kda_conv_fwd(x, weight, bias=None, initial_state=None, *, activation=None,
                 output_final_state=False, cu_seqlens=None, y=None, stream=None):
    """Returns (y, final_state).

    x [B, T, D] bf16/fp16/fp32, its rows evenly spaced (a column slice of a wider tensor will do);
    weight [D, W], W 2 to 4, and bias [D] (None: zeros) in x's dtype or fp32; ``activation`` None or
    "silu".  initial_state [sequences, W - 1, D] (x's dtype) are the inputs in front of each
    sequence, oldest first (None: zeros); final_state, the last W - 1 of state and sequence, is
    None unless ``output_final_state``.  ``cu_seqlens`` (int32 [N + 1] on the device, B = 1) packs N
    sequences along T; y is zero at tokens in no sequence when it is allocated here.
    """
    if stream is None and y is None and activation in _ALLOWED:
        out = library().quick_conv_fwd(x, weight, bias, initial_state, activation is not None,
                                       output_final_state, cu_seqlens)
        if out is not None:
            return out
    return _conv_fwd(x, weight, bias, initial_state, activation, output_final_state, cu_seqlens, y,
                     stream=stream)


@takes_stream
def _conv_fwd(x, weight, bias, initial_state, activation, output_final_state, cu_seqlens, y):
    D, W, dev, wdtype = _inputs("kda_conv_fwd", x, weight, bias, 2)
    act = activation_code(activation, _ALLOWED)
    B, T, dt = x.shape[0], x.shape[1], x.dtype
    N = sequences(cu_seqlens, B, dev)
    op = ConvFwdOpts(x_stride=row_stride("x", x, x.shape, dt, dev))
    if y is None:
        y = torch.empty(x.shape, dtype=dt, device=x.device)
        op.zero_rest = 1
    else:
        op.y_stride = row_stride("y", y, x.shape, dt, dev)
    if N:
        op.num_seqs, op.cu_seqlens = N, cu_seqlens.data_ptr()
    if initial_state is not None:
        check("initial_state", initial_state, (N or B, W - 1, D), dt, dev)
        op.initial_state = initial_state.data_ptr()
    final = None
    if output_final_state:
        final = torch.empty((N or B, W - 1, D), dtype=dt, device=x.device)
        op.final_state = final.data_ptr()
    if B:
        run("kda_conv_fwd", dev, x.data_ptr(), weight.data_ptr(), ptr(bias), y.data_ptr(), B, T, D, W,
            DTYPES[dt], wdtype, act, ctypes.addressof(op))
    return y, final


def kda_conv_bwd(dy, x, weight, bias=None, initial_state=None, d_final_state=None, *, activation=None,
                 output_d_initial_state=False, cu_seqlens=None, dx=None, param_grads=True, stream=None):
    """Gradients of ``kda_conv_fwd``.  Returns (dx, dweight, dbias, d_initial_state).

    x, the parameters, initial_state, ``activation`` and ``cu_seqlens`` as given to the forward, dy
    like its y.  dx is in x's dtype; dweight [D, W] and dbias [D] are fp32, summed over the tokens
    in a fixed order (None unless ``param_grads``).  d_final_state (None: zeros) and d_initial_state
    (None unless ``output_d_initial_state``) are like the states.
    """
    if (stream is None and initial_state is None and d_final_state is None
            and not output_d_initial_state and dx is None and param_grads and activation in _ALLOWED):
        out = library().quick_conv_bwd(dy, x, weight, bias, activation is not None, cu_seqlens)
        if out is not None:
            return out
    return _conv_bwd(dy, x, weight, bias, initial_state, d_final_state, activation,
                     output_d_initial_state, cu_seqlens, dx, param_grads, stream=stream)


@takes_stream
def _conv_bwd(dy, x, weight, bias, initial_state, d_final_state, activation, output_d_initial_state,
              cu_seqlens, dx, param_grads):
    D, W, dev, wdtype = _inputs("kda_conv_bwd", x, weight, bias, 2)
    act = activation_code(activation, _ALLOWED)
    B, T, dt = x.shape[0], x.shape[1], x.dtype
    N = sequences(cu_seqlens, B, dev)
    op = ConvBwdOpts(x_stride=row_stride("x", x, x.shape, dt, dev),
                     dy_stride=row_stride("dy", dy, x.shape, dt, dev))
    if dx is None:
        dx = torch.empty(x.shape, dtype=dt, device=x.device)
        op.zero_rest = 1
    else:
        op.dx_stride = row_stride("dx", dx, x.shape, dt, dev)
    if N:
        op.num_seqs, op.cu_seqlens = N, cu_seqlens.data_ptr()
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            check(name, t, (N or B, W - 1, D), dt, dev)
            setattr(op, name, t.data_ptr())
    d_initial = dw = db = None
    if output_d_initial_state:
        d_initial = torch.empty((N or B, W - 1, D), dtype=dt, device=x.device)
        op.d_initial_state = d_initial.data_ptr()
    if param_grads:
        new = torch.empty if B else torch.zeros
        dw = new((D, W), dtype=F32, device=x.device)
        db = new(D, dtype=F32, device=x.device)
        size = library().kda_conv_bwd_workspace_bytes(B, T, D, W, N)
        ws = torch.empty(size, dtype=torch.uint8, device=x.device)
        op.workspace, op.workspace_bytes = ws.data_ptr(), size
    if B:
        run("kda_conv_bwd", dev, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), ptr(bias), dx.data_ptr(),
            ptr(dw), ptr(db), B, T, D, W, DTYPES[dt], wdtype, act, ctypes.addressof(op))
    return dx, dw, db, d_initial


def kda_conv_step(x, state, weight, bias=None, *, activation=None, state_indices=None, y=None,
                  stream=None):
    """One token for each of N requests, the last inputs updated in place.  Returns y [N, D].

    x [N, D], the parameters and ``activation`` as in ``kda_conv_fwd``; state [N, W - 1, D] of x's
    dtype -- or, with ``state_indices`` (int32 [N] on the device), [num_states, ...], request n's
    being state[state_indices[n]].  An index outside the states marks a padding row (its y is zero);
    no two rows may name one state.
    """
    if stream is None and y is None and activation in _ALLOWED:
        out = library().quick_conv_step(x, state, weight, bias, activation is not None, state_indices)
        if out is not None:
            return out
    return _conv_step(x, state, weight, bias, activation, state_indices, y, stream=stream)


@takes_stream
def _conv_step(x, state, weight, bias, activation, state_indices, y):
    D, W, dev, wdtype = _inputs("kda_conv_step", x, weight, bias, 1)
    act = activation_code(activation, _ALLOWED)
    N, dt = x.shape[0], x.dtype
    states = state.shape[0]
    check("state", state, (N if state_indices is None else states, W - 1, D), dt, dev)
    op = ConvStepOpts(num_states=states, x_stride=row_stride("x", x, x.shape, dt, dev))
    if state_indices is not None:
        check("state_indices", state_indices, (N,), torch.int32, dev)
        op.state_indices = state_indices.data_ptr()
    if y is None:
        y = torch.empty(x.shape, dtype=dt, device=x.device)
    else:
        op.y_stride = row_stride("y", y, x.shape, dt, dev)
    run("kda_conv_step", dev, x.data_ptr(), weight.data_ptr(), ptr(bias), state.data_ptr(),
        y.data_ptr(), N, D, W, DTYPES[dt], wdtype, act, ctypes.addressof(op))
    return y
