"""Checks and calls shared by the bindings of the per-channel operators (ssm,
shortconv, groupnorm): argument marshalling only."""
from __future__ import annotations

import torch

from .wkv7 import Wkv7Error, load_library

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_NAMES = {"f32": torch.float32, "bf16": torch.bfloat16}


def dtype_code(t) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return code


def dtype_named(name, default):
    """The torch dtype of "f32" / "bf16" (None: the default)."""
    if name is None:
        return default
    if name not in _NAMES:
        raise ValueError(f"y_dtype must be one of {sorted(_NAMES)}")
    return _NAMES[name]


def check(name, t, shape, dtype, dev):
    """t is a contiguous tensor of this shape (a tuple) and dtype on dev."""
    if t.shape == shape and t.dtype == dtype and t.device == dev and t.is_contiguous():
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous and on {dev}")


def check_if(name, t, shape, dtype, dev):
    if t is not None:
        check(name, t, shape, dtype, dev)


def gpu(name, t, dims):
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError("inputs must be on a GPU device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {t.device}")
    return t.device


def sizes(*n):
    """The sizes of a descriptor, whose fields are int32 (ctypes would keep the low 32 bits of larger ones)."""
    if max(n) > 0x7FFFFFFF or min(n) < -0x80000000:
        raise ValueError(f"sizes of 2^31 and more are not supported (got {max(n, key=abs)})")
    return n


def ptr(t):
    return None if t is None else t.data_ptr()


def ptrs(*tensors):
    """The addresses of tensors, None for None."""
    return [None if t is None else t.data_ptr() for t in tensors]


def output(name, t, like, y_dtype, dev):
    """The output t, checked, or a new one of like's shape and the named dtype (None: like's)."""
    if t is not None:
        check(name, t, like.shape, dtype_named(y_dtype, t.dtype), dev)
        return t
    if y_dtype is None:
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=dtype_named(y_dtype, None), device=dev)


def gradients(grads, wanted, dev):
    """The output tensors of a backward: for each (key, like, shape, dtype) None where like is, else the
    caller's, checked, or a new one (of like itself where shape is None)."""
    others = set(grads) - {w[0] for w in wanted} if grads else None
    if others:   # a tensor under a name of another's would be left as it was
        raise ValueError(f"grads has no {', '.join(sorted(map(str, others)))}; its keys are {', '.join(w[0] for w in wanted)}")
    out = {}
    for key, like, shape, dtype in wanted:
        given = grads.get(key) if grads else None
        if like is None:
            out[key] = None
        elif given is not None:
            check(f"grads[{key!r}]", given, like.shape if shape is None else shape, like.dtype if dtype is None else dtype, dev)
            out[key] = given
        elif shape is None:
            out[key] = torch.empty_like(like)
        else:
            out[key] = torch.empty(shape, dtype=dtype, device=dev)
    return out


def size(fn, *args) -> int:
    """A size query of the library."""
    n = fn(*args)
    if n < 0:
        raise Wkv7Error(int(-n), fn.__name__, load_library().wkv7_last_error().decode())
    return int(n)


def scratch(workspace, need, dev):
    """The caller's workspace, or one of the needed size, as (pointer, bytes, tensor)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _public_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle and the current device's index, without the wrapper objects
# that torch.cuda's own functions make (2 of the 13 microseconds of a small call), where this
# torch has the names that those functions call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def call(fn, dev, *args):
    """fn(*args, stream) on dev's current stream, with dev the current device."""
    index = dev.index
    if _device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc:
        raise Wkv7Error(rc, fn.__name__, load_library().wkv7_last_error().decode())
