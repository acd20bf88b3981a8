"""What the binding's modules share: checks of arguments, and the call into the library."""

from __future__ import annotations

import ctypes
import functools
import sys
import warnings

import torch

KDA_BF16, KDA_FP16, KDA_FP32 = 0, 1, 2
DTYPES16 = {torch.bfloat16: KDA_BF16, torch.float16: KDA_FP16}
DTYPES = {**DTYPES16, torch.float32: KDA_FP32}
K = 128
F32 = torch.float32

_package = sys.modules[__package__]
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def fits(t, shape, dtype, index):
    """A contiguous tensor of that shape and type on CUDA device `index`."""
    return (t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous())


def check(name, t, shape, dtype, index):
    if fits(t, shape, dtype, index):
        return
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


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


def library():
    """The library in use; lib.quick_<name> is the short way into its functions."""
    return _package._lib or _package.load_library()


def run(name, index, *args):
    """Calls lib.<name>(*args, current stream) on CUDA device `index`; raises on an error."""
    fn = getattr(_package._lib or _package.load_library(), name)
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        raise _package.KdaError(rc, name)


def declare(lib):
    """ctypes signatures of the recurrence, single-token and layer-norm entry points."""
    vp, i, ll, z, f = (ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t,
                       ctypes.c_float)
    for name, res, args in (
            ("kda_chunk_saved_bytes", z, [i] * 6),
            ("kda_chunk_fwd", i, [vp] * 6 + [i] * 4 + [vp, vp]),
            ("kda_chunk_bwd_workspace_bytes", z, [i] * 6 + [z]),
            ("kda_chunk_bwd", i, [vp] * 10 + [i] * 4 + [vp, vp]),
            ("kda_step", i, [vp] * 7 + [i] * 3 + [vp, vp]),
            ("kda_layer_norm_fwd", i, [vp] * 6 + [ll, i, f, i, i, ll, ll, vp]),
            ("kda_layer_norm_bwd_workspace_bytes", z, [ll, i]),
            ("kda_layer_norm_bwd", i, [vp] * 8 + [ll, i, i, i, ll, ll, ll, vp, z, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _declare_quick(lib)


def _declare_quick(lib):
    """The short way in (csrc/binding.cpp) as lib.quick_<name>: functions that return None for
    arguments that need the checks here.  Without _native.so every call goes that way: it takes
    longer (10 us of a small call), and the intra-chunk calls need nothing of it."""

    def address(name):
        return ctypes.cast(getattr(lib, name), ctypes.c_void_p).value

    try:
        from . import _native
    except ImportError as e:
        def quick(name, fns, why=str(e)):
            return lambda *args: _without_native(why)
    else:
        def quick(name, fns):
            return functools.partial(getattr(_native, name), *[address(f) for f in fns])

    for name, fns in (
            ("step", ("kda_step",)),
            ("chunk_fwd", ("kda_chunk_fwd", "kda_chunk_saved_bytes")),
            ("chunk_bwd", ("kda_chunk_bwd", "kda_chunk_saved_bytes",
                           "kda_chunk_bwd_workspace_bytes")),
            ("layer_norm_fwd", ("kda_layer_norm_fwd",)),
            ("layer_norm_bwd", ("kda_layer_norm_bwd", "kda_layer_norm_bwd_workspace_bytes"))):
        setattr(lib, "quick_" + name, quick(name, fns))


@functools.cache
def _without_native(why):
    warnings.warn("_native.so is missing or of another torch: small calls of the recurrence, the "
                  "single-token form and layer norm take longer on the host; build it with "
                  f"gated_delta_rule_intra_gb300.build.build_native() ({why})", RuntimeWarning)
