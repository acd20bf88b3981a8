"""The gated delta-rule recurrence over whole sequences (``kda_chunk_fwd``,
``kda_chunk_bwd``) and its single-token form (``kda_step``).  ``stream=`` (a torch stream or a
raw handle) runs a call on another stream than the current one.

Per value head the state S is [128 dk, 128 dv] in fp32; a token decays it per channel and
corrects it towards its value::

    S~ = diag(2^gate) S,  e = v - S~^T k,  S' = S~ + beta k e^T,  o = scale S'^T q
"""

from __future__ import annotations

import ctypes

import torch

from ._common import DTYPES16, F32, K, check, fits, library, run, takes_stream


class ChunkFwdOpts(ctypes.Structure):
    """Mirror of kda_chunk_fwd_opts_t."""
    _fields_ = [("HV", ctypes.c_int), ("scale", ctypes.c_float),
                ("initial_state", ctypes.c_void_p), ("final_state", ctypes.c_void_p),
                ("saved", ctypes.c_void_p), ("saved_bytes", ctypes.c_size_t),
                ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("zero_rest", ctypes.c_int)]


class ChunkBwdOpts(ctypes.Structure):
    """Mirror of kda_chunk_bwd_opts_t."""
    _fields_ = [("HV", ctypes.c_int), ("scale", ctypes.c_float),
                ("d_final_state", ctypes.c_void_p), ("d_initial_state", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("zero_rest", ctypes.c_int), ("saved", ctypes.c_void_p),
                ("saved_bytes", ctypes.c_size_t), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class StepOpts(ctypes.Structure):
    """Mirror of kda_step_opts_t."""
    _fields_ = [("HV", ctypes.c_int), ("scale", ctypes.c_float),
                ("state_indices", ctypes.c_void_p), ("num_states", ctypes.c_int)]


def _inputs(fn, q, k, v, gate, beta, lead):
    """Checks of the five inputs; (H, HV, device index)."""
    shape, vshape, dt, dev = q.shape, v.shape, q.dtype, q.get_device()
    if (len(shape) == lead + 2 == len(vshape) and shape[-1] == K and dt in DTYPES16 and dev >= 0
            and shape[lead] and vshape[lead] % shape[lead] == 0
            and fits(q, shape, dt, dev) and fits(k, shape, dt, dev)
            and fits(v, (*shape[:lead], vshape[lead], K), dt, dev) and fits(gate, vshape, F32, dev)
            and fits(beta, vshape[:-1], F32, dev)):
        return shape[lead], vshape[lead], dev
    if dev < 0:
        raise ValueError(f"{fn} needs CUDA tensors (no CPU path exists)")
    if dt not in DTYPES16:
        raise ValueError(f"q/k/v dtype must be bf16 or fp16, got {dt}")
    rows = "N" if lead == 1 else "B, T"
    if len(shape) != lead + 2 or shape[-1] != K:
        raise ValueError(f"q must be [{rows}, H, {K}], got {tuple(shape)}")
    if len(vshape) != lead + 2:
        raise ValueError(f"v must be [{rows}, HV, {K}], got {tuple(vshape)}")
    H, HV = shape[lead], vshape[lead]
    if H == 0 or HV % H:
        raise ValueError(f"v's {HV} heads must be a multiple of q's {H}")
    check("q", q, shape, dt, dev)
    check("k", k, shape, dt, dev)
    check("v", v, (*shape[:lead], HV, K), dt, dev)
    check("gate", gate, vshape, F32, dev)
    check("beta", beta, vshape[:-1], F32, dev)
    raise AssertionError("unreachable")


def _scale(scale):
    if scale is None:
        return 0.0  # the library's default
    if scale == 0:
        raise ValueError("scale must not be 0")
    return float(scale)


def _seqs(cu_seqlens, B, dev):
    if cu_seqlens is None:
        return 0
    if B != 1:
        raise ValueError("cu_seqlens packs sequences along T: B must be 1")
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must have at least two entries")
    check("cu_seqlens", cu_seqlens, (cu_seqlens.numel(),), torch.int32, dev)
    return cu_seqlens.numel() - 1


def kda_chunk_fwd(q, k, v, gate, beta, scale=None, initial_state=None, *,
                  output_final_state=False, save=False, cu_seqlens=None, o=None, precise=False,
                  stream=None):
    """The recurrence over whole sequences.  Returns (o, final_state, saved).

    q, k [B, T, H, 128] and v [B, T, HV, 128] bf16/fp16 (value head hv reads q/k head
    hv // (HV // H)); gate [B, T, HV, 128] fp32 per-step log2 decays, <= 0 (not cumulative);
    beta [B, T, HV] fp32; any T.  ``scale`` defaults to 128 ** -0.5.  ``initial_state``
    [sequences, HV, 128 dk, 128 dv] fp32 defaults to zeros.  o is in q's dtype, with zeros at
    tokens in no sequence when it is allocated here.  final_state (fp32) is None unless
    ``output_final_state``.  saved is what ``kda_chunk_bwd`` needs (0.9 KB a token and
    value head in bf16 without a state, 1.7 KB otherwise), None unless ``save``.  bf16 calls
    without a state take fp16 operands of 11 bits (o within 1e-3 beside its rounding) unless
    ``precise``; all others keep 16 bits and more (1e-5).
    ``cu_seqlens`` (int32 [N + 1] on the device, B = 1) packs N sequences along T; it is read on
    the device only.
    """
    if stream is None and cu_seqlens is None and o is None and not precise:
        out = library().quick_chunk_fwd(q, k, v, gate, beta, scale, initial_state,
                                        output_final_state, save)
        if out is not None:
            return out
    return _chunk_fwd(q, k, v, gate, beta, scale, initial_state, output_final_state, save,
                      cu_seqlens, o, precise, stream=stream)


@takes_stream
def _chunk_fwd(q, k, v, gate, beta, scale, initial_state, output_final_state, save, cu_seqlens, o,
               precise=False):
    H, HV, dev = _inputs("kda_chunk_fwd", q, k, v, gate, beta, 2)
    B, T = q.shape[:2]
    N = _seqs(cu_seqlens, B, dev)
    op = ChunkFwdOpts(HV=HV, scale=_scale(scale))
    if o is None:
        o = torch.empty_like(v)
        op.zero_rest = 1
    else:
        check("o", o, v.shape, v.dtype, dev)
    if N:
        op.num_seqs, op.cu_seqlens = N, cu_seqlens.data_ptr()
    if initial_state is not None:
        check("initial_state", initial_state, (N or B, HV, K, K), F32, dev)
        op.initial_state = initial_state.data_ptr()
    final = saved = None
    if output_final_state or (precise and not save):  # taking a state is what asks for it there
        final = torch.empty((N or B, HV, K, K), dtype=F32, device=q.device)
        op.final_state = final.data_ptr()
    if save:
        size = library().kda_chunk_saved_bytes(B, T, HV, N, DTYPES16[q.dtype],
                                               initial_state is not None or output_final_state
                                               or precise)
        saved = torch.empty(size, dtype=torch.uint8, device=q.device)
        op.saved, op.saved_bytes = saved.data_ptr(), size
    if B:
        run("kda_chunk_fwd", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), gate.data_ptr(),
            beta.data_ptr(), o.data_ptr(), B, T, H, DTYPES16[q.dtype], ctypes.addressof(op))
    return o, final if output_final_state else None, saved


def kda_chunk_bwd(q, k, v, gate, beta, do, saved, scale=None, d_final_state=None, *,
                  output_d_initial_state=False, cu_seqlens=None, dq=None, dk=None, dv=None,
                  dgate=None, dbeta=None, gate_grads_fp32=False, stream=None):
    """Gradients of ``kda_chunk_fwd``.  Returns (dq, dk, dv, dgate, dbeta, d_initial_state).

    The five inputs, ``scale`` and ``cu_seqlens`` as given to the forward, do like its o,
    ``saved`` what it returned with ``save=True`` (read only).  The gradients are in q's dtype,
    dgate and dbeta in fp32 with ``gate_grads_fp32`` (as gate and beta themselves are); dq and
    dk are summed over the value heads of their head.  ``d_final_state`` (fp32, the final
    state's shape) defaults to zeros; d_initial_state (fp32) is None unless
    ``output_d_initial_state``.  Deterministic.
    """
    if (stream is None and cu_seqlens is None and d_final_state is None
            and not output_d_initial_state and dq is None and dk is None and dv is None
            and dgate is None and dbeta is None and not gate_grads_fp32):
        out = library().quick_chunk_bwd(q, k, v, gate, beta, do, saved, scale)
        if out is not None:
            return out
    return _chunk_bwd(q, k, v, gate, beta, do, saved, scale, d_final_state,
                      output_d_initial_state, cu_seqlens, (dq, dk, dv, dgate, dbeta),
                      gate_grads_fp32, stream=stream)


@takes_stream
def _chunk_bwd(q, k, v, gate, beta, do, saved, scale, d_final_state, output_d_initial_state,
               cu_seqlens, given, gate_grads_fp32=False):
    H, HV, dev = _inputs("kda_chunk_bwd", q, k, v, gate, beta, 2)
    B, T, dt = q.shape[0], q.shape[1], q.dtype
    N = _seqs(cu_seqlens, B, dev)
    check("do", do, v.shape, dt, dev)
    lib = library()
    saved_bytes = saved.numel()
    if saved_bytes not in (lib.kda_chunk_saved_bytes(B, T, HV, N, DTYPES16[dt], 0),
                           lib.kda_chunk_saved_bytes(B, T, HV, N, DTYPES16[dt], 1)):
        raise ValueError(f"saved has {saved_bytes} bytes: not from a forward of these inputs")
    check("saved", saved, (saved_bytes,), torch.uint8, dev)
    zero_rest = all(t is None for t in given)
    new = torch.zeros_like if N and not zero_rest else torch.empty_like
    out = []
    gdt = F32 if gate_grads_fp32 else dt
    for name, t, like, ty in zip(("dq", "dk", "dv", "dgate", "dbeta"), given,
                                 (q, k, v, gate, beta), (dt, dt, dt, gdt, gdt)):
        if t is None:
            t = new(like, dtype=ty)
        else:
            check(name, t, like.shape, ty, dev)
        out.append(t)
    op = ChunkBwdOpts(HV=HV, scale=_scale(scale), saved=saved.data_ptr(), saved_bytes=saved_bytes,
                      zero_rest=zero_rest + (2 if gate_grads_fp32 else 0))
    if N:
        op.num_seqs, op.cu_seqlens = N, cu_seqlens.data_ptr()
    if d_final_state is not None:
        check("d_final_state", d_final_state, (N or B, HV, K, K), F32, dev)
        op.d_final_state = d_final_state.data_ptr()
    d_initial = None
    if output_d_initial_state:
        d_initial = torch.empty((N or B, HV, K, K), dtype=F32, device=q.device)
        op.d_initial_state = d_initial.data_ptr()
    if B:
        work = lib.kda_chunk_bwd_workspace_bytes(B, T, H, HV, N, DTYPES16[dt], saved_bytes)
        ws = torch.empty(work, dtype=torch.uint8, device=q.device)
        op.workspace, op.workspace_bytes = ws.data_ptr(), work
        run("kda_chunk_bwd", dev, q.data_ptr(), k.data_ptr(), gate.data_ptr(), beta.data_ptr(),
            do.data_ptr(), *[t.data_ptr() for t in out], B, T, H, DTYPES16[dt],
            ctypes.addressof(op))
    return (*out, d_initial)


def kda_step(q, k, v, gate, beta, state, scale=None, *, state_indices=None, o=None, stream=None):
    """One token for each of N requests, the states updated in place.  Returns o [N, HV, 128].

    q, k [N, H, 128], v [N, HV, 128] bf16/fp16, gate [N, HV, 128] and beta [N, HV] fp32 as in
    ``kda_chunk_fwd``; state [N, HV, 128 dk, 128 dv] fp32 -- or, with ``state_indices`` (int32
    [N] on the device), [num_states, ...], request n's being state[state_indices[n]].  An index
    outside the states marks a padding row (its o is zero); no two rows may name one state.
    """
    if stream is None:
        out = library().quick_step(q, k, v, gate, beta, state, scale, state_indices, o)
        if out is not None:
            return out
    return _step(q, k, v, gate, beta, state, scale, state_indices, o, stream=stream)


@takes_stream
def _step(q, k, v, gate, beta, state, scale, state_indices, o):
    H, HV, dev = _inputs("kda_step", q, k, v, gate, beta, 1)
    N, states = q.shape[0], state.shape[0]
    check("state", state, (N if state_indices is None else states, HV, K, K), F32, dev)
    op = StepOpts(HV=HV, scale=_scale(scale), num_states=states)
    if state_indices is not None:
        check("state_indices", state_indices, (N,), torch.int32, dev)
        op.state_indices = state_indices.data_ptr()
    if o is None:
        o = torch.empty_like(v)
    else:
        check("o", o, v.shape, v.dtype, dev)
    run("kda_step", dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), gate.data_ptr(),
        beta.data_ptr(), state.data_ptr(), o.data_ptr(), N, H, DTYPES16[q.dtype],
        ctypes.addressof(op))
    return o
