"""What the binding's modules share: checks of arguments, and the current stream."""

from __future__ import annotations

import ctypes
import functools

import torch

KDA_BF16, KDA_FP16, KDA_FP32 = 0, 1, 2
DTYPES16 = {torch.bfloat16: KDA_BF16, torch.float16: KDA_FP16}
DTYPES = {**DTYPES16, torch.float32: KDA_FP32}
K = 128
F32 = torch.float32


def check(name, t, shape, dtype, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def ptr(t):
    return None if t is None else t.data_ptr()


def takes_stream(fn):
    """Adds ``stream=`` (a torch stream or a raw handle; default: the current one).  The call
    then runs with that stream current, so that what it allocates -- outputs, workspaces --
    belongs to the stream that uses it."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=args[0].device)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)

    return call


def run(name, device, *args):
    """Calls lib.<name>(*args, current stream) on the tensors' device; raises on an error."""
    from . import KdaError, load_library
    index = device.index
    fn = getattr(load_library(), name)
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc:
        raise KdaError(rc, name)


def declare(lib):
    """ctypes signatures of the recurrence, single-token and layer-norm entry points."""
    vp, i, ll, z, f = (ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t,
                       ctypes.c_float)
    for name, res, args in (
            ("kda_chunk_saved_bytes", z, [i] * 4),
            ("kda_chunk_fwd", i, [vp] * 6 + [i] * 4 + [vp, vp]),
            ("kda_chunk_bwd_workspace_bytes", z, [i] * 5),
            ("kda_chunk_bwd", i, [vp] * 10 + [i] * 4 + [vp, vp]),
            ("kda_step", i, [vp] * 7 + [i] * 3 + [vp, vp]),
            ("kda_layer_norm_fwd", i, [vp] * 6 + [ll, i, f, i, i, ll, ll, vp]),
            ("kda_layer_norm_bwd_workspace_bytes", z, [ll, i]),
            ("kda_layer_norm_bwd", i, [vp] * 8 + [ll, i, i, i, ll, ll, ll, vp, z, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
