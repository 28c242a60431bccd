"""Binding of linear attention with a decay for each head (include/linattn.h) on torch
GPU tensors: linattn_forward, linattn_step, linattn_backward.  Argument marshalling
only; without the library every call raises.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,  y_t = scale S_t^T q_t      per head

Shapes: q [B, T, Hq, Dk], k [B, T, Hk, Dk], v [B, T, Hv, Dv] float32 or bfloat16; g float32
[B, T, H], or [H] for constant decays; y [B, T, H, Dv]; states [B, H, Dk, Dv] float32;
lengths [B] int32.  Hq, Hk and Hv divide H: consecutive heads share one.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _marshal as M
from .wkv7 import load_library

__all__ = ["linattn_forward", "linattn_step", "linattn_backward", "linattn_workspace_bytes", "linattn_backward_workspace_bytes",
           "LinattnDesc", "EXPORTED_SYMBOLS"]

EXPORTED_SYMBOLS = ("linattn_workspace_bytes", "linattn_forward", "linattn_step", "linattn_backward_workspace_bytes", "linattn_backward")


class LinattnDesc(ctypes.Structure):
    """Mirror of struct linattn_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "H", "Hq", "Hk", "Hv", "Dk", "Dv", "in_dtype", "y_dtype", "g_per_token", "S")] + \
               [("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("lengths", ctypes.c_void_p)]


_FN = None


def _lib():
    """The library with these functions' signatures declared (once)."""
    global _FN
    if _FN is None:
        lib = load_library()
        d, vp, i64 = ctypes.POINTER(LinattnDesc), ctypes.c_void_p, ctypes.c_int64
        for name, args, res in (("linattn_workspace_bytes", [d], i64),
                                ("linattn_forward", [d] + [vp] * 8 + [i64, vp], ctypes.c_int),
                                ("linattn_step", [d] + [vp] * 8, ctypes.c_int),
                                ("linattn_backward_workspace_bytes", [d], i64),
                                ("linattn_backward", [d] + [vp] * 13 + [i64, vp], ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _FN = lib
    return _FN


def _sizes(B, T, H, Dk, Dv, Hq, Hk, Hv, dtype):
    M.sizes(B, T, H, Dk, Dv, Hq, Hk, Hv)
    return LinattnDesc(B, T, H, Hq, Hk, Hv, Dk, Dv, dtype, dtype, 1, 0, 1.0, 0, None)


def linattn_workspace_bytes(B: int, T: int, H: int, Dk: int, Dv: int, *, Hq: int = 0, Hk: int = 0, Hv: int = 0) -> int:
    """Workspace bytes of linattn_forward for these sizes, of either dtype."""
    return max(M.size(_lib().linattn_workspace_bytes, ctypes.byref(_sizes(B, T, H, Dk, Dv, Hq, Hk, Hv, d))) for d in (0, 1))


def linattn_backward_workspace_bytes(B: int, T: int, H: int, Dk: int, Dv: int, *, Hq: int = 0, Hk: int = 0, Hv: int = 0) -> int:
    """Workspace bytes of linattn_backward for these sizes, of either dtype."""
    return max(M.size(_lib().linattn_backward_workspace_bytes, ctypes.byref(_sizes(B, T, H, Dk, Dv, Hq, Hk, Hv, d))) for d in (0, 1))


def _inputs(q, k, v, g, lengths, step):
    """Check the inputs; the device and the sizes."""
    dims = 3 if step else 4
    dev = M.gpu("q", q, dims)
    row, Hq, Dk = q.shape[:-2], q.shape[-2], q.shape[-1]
    for name, t in (("k", k), ("v", v)):
        if t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    Hk, Hv, Dv = k.shape[-2], v.shape[-2], v.shape[-1]
    M.check("k", k, row + (Hk, Dk), q.dtype, dev)
    M.check("v", v, row + (Hv, Dv), q.dtype, dev)
    if g.dim() not in (1, len(row) + 1):
        raise ValueError(f"g must be [H] or {'[B, H]' if step else '[B, T, H]'}, got {tuple(g.shape)}")
    H = g.shape[-1]
    M.check("g", g, (H,) if g.dim() == 1 else row + (H,), torch.float32, dev)
    if (H == 0) != (Hq == 0) or any(n == 0 or H % n for n in (Hq, Hk, Hv) if H):
        raise ValueError(f"{Hq}, {Hk} and {Hv} heads of q, k and v must divide the {H} of g")
    M.check_if("lengths", lengths, row[:1], torch.int32, dev)
    return dev, row[0], 1 if step else row[1], H, Hq, Hk, Hv, Dk, Dv


def _desc(q, y, g, n, scale, lengths=None, S=0):
    _, B, T, H, Hq, Hk, Hv, Dk, Dv = n
    M.sizes(B, T, H, Hq, Hk, Hv, Dk, Dv, S)
    return LinattnDesc(B, T, H, Hq, Hk, Hv, Dk, Dv, M.dtype_code(q), M.dtype_code(y), 0 if g.dim() == 1 else 1, S, scale, 0, M.ptr(lengths))


def _output(y, v, shape, y_dtype, dev):
    if y is not None:
        M.check("y", y, shape, M.dtype_named(y_dtype, y.dtype), dev)
        return y
    return torch.empty(shape, dtype=M.dtype_named(y_dtype, v.dtype), device=dev)


def linattn_forward(q, k, v, g, *, scale: float = 1.0, state=None, lengths=None, y_dtype: Optional[str] = None, y=None,
                    state_out=None, return_state: bool = True, workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The recurrence over T tokens from `state` (None: zeros).  Returns (y, state_out); outputs
    are allocated unless given (state_out may be state: in place), state_out is None when
    return_state is False.  lengths: tokens of each sequence (the others are padding: y 0,
    state untouched)."""
    n = dev, B, T, H, _, _, _, Dk, Dv = _inputs(q, k, v, g, lengths, False)
    st = (B, H, Dk, Dv)
    M.check_if("state", state, st, torch.float32, dev)
    y = _output(y, v, (B, T, H, Dv), y_dtype, dev)
    if state_out is not None:
        M.check("state_out", state_out, st, torch.float32, dev)
    elif return_state:
        state_out = torch.empty(st, dtype=torch.float32, device=dev)
    desc = _desc(q, y, g, n, scale, lengths)
    lib = _lib()
    ws, ws_bytes, keep = M.scratch(workspace, M.size(lib.linattn_workspace_bytes, ctypes.byref(desc)), dev)
    M.call(lib.linattn_forward, dev, ctypes.byref(desc), *M.ptrs(q, k, v, g, state, y, state_out), ws, ws_bytes)
    return y, state_out


def linattn_step(q, k, v, g, state, *, scale: float = 1.0, state_index=None, y_dtype: Optional[str] = None, y=None) -> torch.Tensor:
    """One token per row: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hv, Dv], g [B, H] or [H], state
    [S, H, Dk, Dv] updated in place; returns y [B, H, Dv].  Row b works on state state_index[b]
    (int32 [B]; None: state b).  A row whose index is outside 0 .. S - 1, or that an earlier row
    already names, has no request: its y is 0 and no state changes for it."""
    n = dev, B, _, H, _, _, _, Dk, Dv = _inputs(q, k, v, g, None, True)
    S = state.shape[0] if state.dim() else 0
    M.check("state", state, (S, H, Dk, Dv), torch.float32, dev)
    M.check_if("state_index", state_index, (B,), torch.int32, dev)
    y = _output(y, v, (B, H, Dv), y_dtype, dev)
    desc = _desc(q, y, g, n, scale, None, S)
    M.call(_lib().linattn_step, dev, ctypes.byref(desc), *M.ptrs(q, k, v, g, state, state_index, y))
    return y


def linattn_backward(q, k, v, g, dy, *, scale: float = 1.0, state=None, dstate=None, lengths=None, workspace=None, grads=None,
                     return_dg: bool = True, return_dstate: bool = True) -> dict:
    """Gradients of <dy, y> + <dstate, state_out> for linattn_forward with the same arguments.

    dy [B, T, H, Dv] of the y dtype; dstate [B, H, Dk, Dv] float32 or None.  Returns a dict: q,
    k, v of the input dtype, g as g (None when return_dg is False), state [B, H, Dk, Dv] float32
    (None when return_dstate is False).  `grads` may supply output tensors under these keys
    (others: ValueError)."""
    n = dev, B, T, H, _, _, _, Dk, Dv = _inputs(q, k, v, g, lengths, False)
    st = (B, H, Dk, Dv)
    M.check_if("state", state, st, torch.float32, dev)
    M.check("dy", dy, (B, T, H, Dv), dy.dtype, dev)
    M.check_if("dstate", dstate, st, torch.float32, dev)
    out = M.gradients(grads, (("q", q, None, None), ("k", k, None, None), ("v", v, None, None), ("g", g if return_dg else None, None, None),
                              ("state", q if return_dstate else None, st, torch.float32)), dev)
    desc = _desc(q, dy, g, n, scale, lengths)
    lib = _lib()
    ws, ws_bytes, keep = M.scratch(workspace, M.size(lib.linattn_backward_workspace_bytes, ctypes.byref(desc)), dev)
    M.call(lib.linattn_backward, dev, ctypes.byref(desc),
           *M.ptrs(q, k, v, g, state, dy, dstate, out["q"], out["k"], out["v"], out["g"], out["state"]), ws, ws_bytes)
    return out
