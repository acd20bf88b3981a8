"""The selective state-space scan over whole sequences (``kda_scan_fwd``, ``kda_scan_bwd``) and its
single-token form (``kda_scan_step``).  ``stream=`` (a torch stream or a raw handle) runs a call on
another stream than the current one.

Per channel a state h of N numbers in fp32; with s = softplus(delta + delta_bias)::

    h' = exp(s A) h + s u B,  y = (sum_n C h' + D u) silu(z)
"""

from __future__ import annotations

import ctypes

import torch

from ._common import DTYPES, F32, check, library, ptr, row_stride, run, sequences, takes_stream

MAX_STATES = 64


class ScanFwdOpts(ctypes.Structure):
    """Mirror of kda_scan_fwd_opts_t."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("skip", "delta_bias", "z", "initial_state",
                                                "final_state", "saved")]
                + [("saved_bytes", ctypes.c_size_t), ("cu_seqlens", ctypes.c_void_p)]
                + [(n, ctypes.c_int) for n in ("num_seqs", "zero_rest", "plain_delta")]
                + [(n + "_stride", ctypes.c_longlong) for n in ("u", "delta", "z", "B", "C", "y")]
                + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)])


class ScanBwdOpts(ctypes.Structure):
    """Mirror of kda_scan_bwd_opts_t."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("skip", "delta_bias", "z", "dskip", "ddelta_bias",
                                                "dz", "d_final_state", "d_initial_state", "saved")]
                + [("saved_bytes", ctypes.c_size_t), ("cu_seqlens", ctypes.c_void_p)]
                + [(n, ctypes.c_int) for n in ("num_seqs", "zero_rest", "plain_delta")]
                + [(n + "_stride", ctypes.c_longlong) for n in ("dy", "u", "delta", "z", "B", "C")]
                + [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)])


class ScanStepOpts(ctypes.Structure):
    """Mirror of kda_scan_step_opts_t."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("skip", "delta_bias", "z", "state_indices")]
                + [(n, ctypes.c_int) for n in ("num_states", "plain_delta")]
                + [(n + "_stride", ctypes.c_longlong) for n in ("u", "delta", "z", "B", "C", "y")])


def _inputs(fn, op, u, delta, A, B, C, D, z, delta_bias, lead):
    """Checks of the inputs, whose strides and pointers go into `op`; (D, N, G, device index)."""
    dev, shape, dt = u.get_device(), u.shape, u.dtype
    if dev < 0:
        raise ValueError(f"{fn} needs CUDA tensors (no CPU path exists)")
    if dt not in DTYPES:
        raise ValueError(f"u must be bf16, fp16 or fp32, got {dt}")
    rows = "N" if lead == 1 else "B, T"
    if len(shape) != lead + 1 or shape[-1] == 0:
        raise ValueError(f"u must be [{rows}, D], got {tuple(shape)}")
    width = shape[-1]
    if A.dim() != 2 or A.shape[0] != width or not 1 <= A.shape[1] <= MAX_STATES:
        raise ValueError(f"A must be [{width}, states] with 1 to {MAX_STATES} states, got "
                         f"{tuple(A.shape)}")
    N = A.shape[1]
    check("A", A, A.shape, F32, dev)
    if B.dim() != lead + 2 or B.shape[-2] == 0 or width % B.shape[-2]:
        raise ValueError(f"B must be [{rows}, groups, {N}] with groups a divisor of {width}, got "
                         f"{tuple(B.shape)}")
    G = B.shape[-2]
    vec = (*shape[:-1], G, N)
    op.u_stride = row_stride("u", u, shape, dt, dev)
    op.delta_stride = row_stride("delta", delta, shape, dt, dev)
    op.B_stride = row_stride("B", B, vec, dt, dev, 2)
    op.C_stride = row_stride("C", C, vec, dt, dev, 2)
    if z is not None:
        op.z_stride, op.z = row_stride("z", z, shape, dt, dev), z.data_ptr()
    for name, field, t in (("D", "skip", D), ("delta_bias", "delta_bias", delta_bias)):
        if t is not None:
            check(name, t, (width,), F32, dev)
            setattr(op, field, t.data_ptr())
    return width, N, G, dev


def kda_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, initial_state=None, *,
                 delta_softplus=True, output_final_state=False, save=False, cu_seqlens=None, y=None,
                 stream=None):
    """The scan over whole sequences.  Returns (y, final_state, saved).

    u, delta, z [B, T, D] and B, C [B, T, groups, N] bf16/fp16/fp32 (one dtype), N up to 64, their
    rows evenly spaced (column slices of wider tensors will do); channel d reads group
    d // (D // groups).  A [D, N], D [D] (the skip) and delta_bias [D] fp32.  D, z and delta_bias
    may be None; without ``delta_softplus`` the step sizes are delta + delta_bias as they are.
    ``initial_state`` [sequences, D, N] fp32 defaults to zeros; final_state is None unless
    ``output_final_state``; saved is what ``kda_scan_bwd`` needs, None unless ``save``: P / 2 + 4 bytes a
    token and channel, P being N rounded up to 8, 16, 32 or 64, with each sequence's tokens rounded up to 16 in
    the first term (packed ones take up to 16 more), the 4 with or without z.  ``cu_seqlens`` (int32 [N + 1]
    on the device, B = 1) packs sequences along T; y is zero at tokens in no sequence when it is allocated
    here.
    """
    if stream is None and y is None and delta_softplus:
        out = library().quick_scan_fwd(u, delta, A, B, C, D, z, delta_bias, initial_state,
                                       output_final_state, save, cu_seqlens)
        if out is not None:
            return out
    return _scan_fwd(u, delta, A, B, C, D, z, delta_bias, initial_state, delta_softplus,
                     output_final_state, save, cu_seqlens, y, stream=stream)


@takes_stream
def _scan_fwd(u, delta, A, B, C, D, z, delta_bias, initial_state, delta_softplus,
              output_final_state, save, cu_seqlens, y):
    op = ScanFwdOpts(plain_delta=not delta_softplus)
    width, N, G, dev = _inputs("kda_scan_fwd", op, u, delta, A, B, C, D, z, delta_bias, 2)
    batch, T, dt = u.shape[0], u.shape[1], u.dtype
    seqs = sequences(cu_seqlens, batch, dev)
    if y is None:
        y = torch.empty(u.shape, dtype=dt, device=u.device)
        op.zero_rest = 1
    else:
        op.y_stride = row_stride("y", y, u.shape, dt, dev)
    if seqs:
        op.num_seqs, op.cu_seqlens = seqs, cu_seqlens.data_ptr()
    states = (seqs or batch, width, N)
    if initial_state is not None:
        check("initial_state", initial_state, states, F32, dev)
        op.initial_state = initial_state.data_ptr()
    final = saved = None
    if output_final_state:
        final = torch.empty(states, dtype=F32, device=u.device)
        op.final_state = final.data_ptr()
    lib = library()
    if save:
        size = lib.kda_scan_saved_bytes(batch, T, width, N, seqs)
        saved = torch.empty(size, dtype=torch.uint8, device=u.device)
        op.saved, op.saved_bytes = saved.data_ptr(), size
    if batch:
        work = lib.kda_scan_fwd_workspace_bytes(batch, T, width, N, G, seqs)
        ws = torch.empty(work, dtype=torch.uint8, device=u.device)
        op.workspace, op.workspace_bytes = ws.data_ptr(), work
        run("kda_scan_fwd", dev, u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(),
            C.data_ptr(), y.data_ptr(), batch, T, width, N, G, DTYPES[dt], ctypes.addressof(op))
    return y, final, saved


def kda_scan_bwd(dy, u, delta, A, B, C, saved, D=None, z=None, delta_bias=None, d_final_state=None, *,
                 delta_softplus=True, output_d_initial_state=False, cu_seqlens=None, stream=None):
    """Gradients of ``kda_scan_fwd``.  Returns (du, ddelta, dA, dB, dC, dD, dz, ddelta_bias,
    d_initial_state).

    The inputs, ``delta_softplus`` and ``cu_seqlens`` as given to the forward, dy like its y, ``saved``
    what it returned with ``save=True`` (read only).  du, ddelta, dB, dC and dz are in u's dtype, zero
    at tokens in no sequence; dA, dD and ddelta_bias are fp32.  dD, dz and ddelta_bias are None where
    the forward had none; d_final_state (fp32, None: zeros) and d_initial_state (None unless
    ``output_d_initial_state``) are like the states.  Deterministic.
    """
    if (stream is None and d_final_state is None and delta_softplus
            and not output_d_initial_state):
        out = library().quick_scan_bwd(dy, u, delta, A, B, C, saved, D, z, delta_bias, cu_seqlens)
        if out is not None:
            return out
    return _scan_bwd(dy, u, delta, A, B, C, saved, D, z, delta_bias, d_final_state, delta_softplus,
                     output_d_initial_state, cu_seqlens, stream=stream)


@takes_stream
def _scan_bwd(dy, u, delta, A, B, C, saved, D, z, delta_bias, d_final_state, delta_softplus,
              output_d_initial_state, cu_seqlens):
    op = ScanBwdOpts(plain_delta=not delta_softplus, zero_rest=1)
    width, N, G, dev = _inputs("kda_scan_bwd", op, u, delta, A, B, C, D, z, delta_bias, 2)
    batch, T, dt = u.shape[0], u.shape[1], u.dtype
    seqs = sequences(cu_seqlens, batch, dev)
    op.dy_stride = row_stride("dy", dy, u.shape, dt, dev)
    lib = library()
    size = lib.kda_scan_saved_bytes(batch, T, width, N, seqs)
    if saved.numel() != size:
        raise ValueError(f"saved has {saved.numel()} bytes: not from a forward of these inputs")
    check("saved", saved, (size,), torch.uint8, dev)
    op.saved, op.saved_bytes = saved.data_ptr(), size
    if seqs:
        op.num_seqs, op.cu_seqlens = seqs, cu_seqlens.data_ptr()

    def new(shape, dtype):
        return (torch.empty if batch else torch.zeros)(shape, dtype=dtype, device=u.device)

    du, dd = new(u.shape, dt), new(u.shape, dt)
    dA, dB, dC = new(A.shape, F32), new(B.shape, dt), new(B.shape, dt)
    dD = dz = dbias = d_initial = None
    if z is not None:
        dz = new(u.shape, dt)
        op.dz = dz.data_ptr()
    if D is not None:
        dD = new(width, F32)
        op.dskip = dD.data_ptr()
    if delta_bias is not None:
        dbias = new(width, F32)
        op.ddelta_bias = dbias.data_ptr()
    states = (seqs or batch, width, N)
    if d_final_state is not None:
        check("d_final_state", d_final_state, states, F32, dev)
        op.d_final_state = d_final_state.data_ptr()
    if output_d_initial_state:
        d_initial = new(states, F32)
        op.d_initial_state = d_initial.data_ptr()
    if batch:
        work = lib.kda_scan_bwd_workspace_bytes(batch, T, width, N, G, seqs)
        ws = torch.empty(work, dtype=torch.uint8, device=u.device)
        op.workspace, op.workspace_bytes = ws.data_ptr(), work
        run("kda_scan_bwd", dev, dy.data_ptr(), u.data_ptr(), delta.data_ptr(), A.data_ptr(),
            B.data_ptr(), C.data_ptr(), du.data_ptr(), dd.data_ptr(), dA.data_ptr(), dB.data_ptr(),
            dC.data_ptr(), batch, T, width, N, G, DTYPES[dt], ctypes.addressof(op))
    return du, dd, dA, dB, dC, dD, dz, dbias, d_initial


def kda_scan_step(u, delta, A, B, C, state, D=None, z=None, delta_bias=None, *, delta_softplus=True,
                  state_indices=None, y=None, stream=None):
    """One token for each of N requests, the states updated in place.  Returns y [N, D].

    u, delta, z [N, D] and B, C [N, groups, states] as in ``kda_scan_fwd``; state [N, D, states]
    fp32 -- or, with ``state_indices`` (int32 [N] on the device), [num_states, ...], request n's
    being state[state_indices[n]].  An index outside the states marks a padding row (its y is zero);
    no two rows may name one state.
    """
    if stream is None and y is None and delta_softplus:
        out = library().quick_scan_step(u, delta, A, B, C, state, D, z, delta_bias, state_indices)
        if out is not None:
            return out
    return _scan_step(u, delta, A, B, C, state, D, z, delta_bias, delta_softplus, state_indices, y,
                      stream=stream)


@takes_stream
def _scan_step(u, delta, A, B, C, state, D, z, delta_bias, delta_softplus, state_indices, y):
    op = ScanStepOpts(plain_delta=not delta_softplus)
    width, N, G, dev = _inputs("kda_scan_step", op, u, delta, A, B, C, D, z, delta_bias, 1)
    rows, dt, states = u.shape[0], u.dtype, state.shape[0]
    check("state", state, (rows if state_indices is None else states, width, N), F32, dev)
    op.num_states = states
    if state_indices is not None:
        check("state_indices", state_indices, (rows,), torch.int32, dev)
        op.state_indices = state_indices.data_ptr()
    if y is None:
        y = torch.empty(u.shape, dtype=dt, device=u.device)
    else:
        op.y_stride = row_stride("y", y, u.shape, dt, dev)
    run("kda_scan_step", dev, u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(),
        C.data_ptr(), state.data_ptr(), y.data_ptr(), rows, width, N, G, DTYPES[dt],
        ctypes.addressof(op))
    return y
