"""Binding of the group norm, channels last (include/groupnorm.h) on torch GPU
tensors: groupnorm_forward, groupnorm_backward.  Argument marshalling only;
without the library every call raises.

    y = act((x - mean) rstd weight + bias) gate,   act "none" or "silu"

with mean and variance over the positions of a sequence and the channels of a
group.  Shapes: x, gate, y [B, T, C]; weight, bias [C] float32; mean, rstd [B, G]
float32; lengths [B] int32.  T = 1 normalises every row by itself: for the heads of a
recurrence's output [batch, tokens, H, D] pass it as [batch * tokens, 1, H * D] with
G = H.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _marshal as M
from .wkv7 import load_library

__all__ = ["groupnorm_forward", "groupnorm_backward", "groupnorm_workspace_bytes", "groupnorm_backward_workspace_bytes",
           "ACTS", "GroupnormDesc", "EXPORTED_SYMBOLS"]

EXPORTED_SYMBOLS = ("groupnorm_workspace_bytes", "groupnorm_forward", "groupnorm_backward_workspace_bytes",
                    "groupnorm_backward")
ACTS = {"none": 0, "silu": 1}


class GroupnormDesc(ctypes.Structure):
    """Mirror of struct groupnorm_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "G", "in_dtype", "y_dtype", "act")] + \
               [("eps", ctypes.c_float), ("lengths", ctypes.c_void_p)]


_FN = None


def _lib():
    """The library with these functions' signatures declared (once)."""
    global _FN
    if _FN is None:
        lib = load_library()
        d, vp, i64 = ctypes.POINTER(GroupnormDesc), ctypes.c_void_p, ctypes.c_int64
        for name, args, res in (("groupnorm_workspace_bytes", [d], i64),
                                ("groupnorm_forward", [d] + [vp] * 8 + [i64, vp], ctypes.c_int),
                                ("groupnorm_backward_workspace_bytes", [d], i64),
                                ("groupnorm_backward", [d] + [vp] * 12 + [i64, vp], ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _FN = lib
    return _FN


def groupnorm_workspace_bytes(B: int, T: int, C: int, G: int) -> int:
    """Workspace bytes of groupnorm_forward for these sizes, of either dtype."""
    return max(M.size(_lib().groupnorm_workspace_bytes, ctypes.byref(GroupnormDesc(*M.sizes(B, T, C, G), d, d, eps=1.0))) for d in (0, 1))


def groupnorm_backward_workspace_bytes(B: int, T: int, C: int, G: int) -> int:
    """Workspace bytes of groupnorm_backward for these sizes, of either dtype."""
    return max(M.size(_lib().groupnorm_backward_workspace_bytes, ctypes.byref(GroupnormDesc(*M.sizes(B, T, C, G), d, d, eps=1.0))) for d in (0, 1))


def _inputs(x, G, weight, bias, gate, lengths):
    dev = M.gpu("x", x, 3)
    B, T, C = x.shape
    if G <= 0 or C % G:
        raise ValueError(f"{C} channels are not a multiple of G = {G}")
    M.check_if("weight", weight, (C,), torch.float32, dev)
    M.check_if("bias", bias, (C,), torch.float32, dev)
    M.check_if("gate", gate, x.shape, x.dtype, dev)
    M.check_if("lengths", lengths, (B,), torch.int32, dev)
    return dev, B, T, C


def _act(act) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    return ACTS[act]


def _desc(x, y, B, T, C, G, act, eps, lengths):
    M.sizes(B, T, C, G)
    return GroupnormDesc(B, T, C, G, M.dtype_code(x), M.dtype_code(y), _act(act), eps, M.ptr(lengths))


def groupnorm_forward(x, G: int, *, weight=None, bias=None, gate=None, act: str = "none", eps: float = 1e-5, lengths=None,
                      y_dtype: Optional[str] = None, y=None, mean=None, rstd=None, return_stats: bool = True,
                      workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Returns (y, mean, rstd); mean and rstd, which groupnorm_backward takes, are None when
    return_stats is False and they are not given."""
    dev, B, T, C = _inputs(x, G, weight, bias, gate, lengths)
    y = M.output("y", y, x, y_dtype, dev)
    if return_stats:
        mean = torch.empty((B, G), dtype=torch.float32, device=dev) if mean is None else mean
        rstd = torch.empty((B, G), dtype=torch.float32, device=dev) if rstd is None else rstd
    M.check_if("mean", mean, (B, G), torch.float32, dev)
    M.check_if("rstd", rstd, (B, G), torch.float32, dev)
    desc = _desc(x, y, B, T, C, G, act, eps, lengths)
    lib = _lib()
    ws, ws_bytes, keep = M.scratch(workspace, M.size(lib.groupnorm_workspace_bytes, ctypes.byref(desc)), dev)
    M.call(lib.groupnorm_forward, dev, ctypes.byref(desc), *M.ptrs(x, weight, bias, gate, y, mean, rstd), ws, ws_bytes)
    return y, mean, rstd


def groupnorm_backward(x, G: int, dy, mean, rstd, *, weight=None, bias=None, gate=None, act: str = "none", lengths=None,
                       workspace=None, grads=None) -> dict:
    """Gradients of <dy, y> for groupnorm_forward with the same arguments, mean and rstd as it
    returned them.  Returns a dict: x and gate of x's dtype, weight and bias [C] float32 (None
    where they are not inputs).  `grads` may supply output tensors under these keys (others: ValueError)."""
    dev, B, T, C = _inputs(x, G, weight, bias, gate, lengths)
    f32 = torch.float32
    M.check("dy", dy, x.shape, dy.dtype, dev)
    M.check("mean", mean, (B, G), f32, dev)
    M.check("rstd", rstd, (B, G), f32, dev)
    out = M.gradients(grads, (("x", x, None, None), ("weight", weight, None, None), ("bias", bias, None, None),
                              ("gate", gate, None, None)), dev)
    desc = _desc(x, dy, B, T, C, G, act, 1.0, lengths)
    lib = _lib()
    ws, ws_bytes, keep = M.scratch(workspace, M.size(lib.groupnorm_backward_workspace_bytes, ctypes.byref(desc)), dev)
    M.call(lib.groupnorm_backward, dev, ctypes.byref(desc),
           *M.ptrs(x, weight, bias, gate, dy, mean, rstd, out["x"], out["weight"], out["bias"], out["gate"]), ws, ws_bytes)
    return out
