"""Binding of the short causal convolution (include/shortconv.h) on torch GPU
tensors: shortconv_forward, shortconv_step, shortconv_backward.  Argument
marshalling only; without the library every call raises.

    y_t = act(bias + sum_k w[:, k] x_{t - K + 1 + k}),   act "none" or "silu"

Shapes: x, y [B, T, C]; w [C, K] float32 (K = 2, 3, 4); bias [C] float32; states
[B, K - 1, C] of x's dtype (the last K - 1 inputs, oldest first); lengths [B] int32.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _marshal as M
from .wkv7 import load_library

__all__ = ["shortconv_forward", "shortconv_step", "shortconv_backward", "shortconv_backward_workspace_bytes", "ACTS",
           "ShortconvDesc", "EXPORTED_SYMBOLS"]

EXPORTED_SYMBOLS = ("shortconv_forward", "shortconv_step", "shortconv_backward_workspace_bytes", "shortconv_backward")
ACTS = {"none": 0, "silu": 1}


class ShortconvDesc(ctypes.Structure):
    """Mirror of struct shortconv_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "K", "in_dtype", "y_dtype", "act", "S")] + \
               [("lengths", ctypes.c_void_p)]


_FN = None


def _lib():
    """The library with these functions' signatures declared (once)."""
    global _FN
    if _FN is None:
        lib = load_library()
        d, vp, i64 = ctypes.POINTER(ShortconvDesc), ctypes.c_void_p, ctypes.c_int64
        for name, args, res in (("shortconv_forward", [d] + [vp] * 7, ctypes.c_int),
                                ("shortconv_step", [d] + [vp] * 7, ctypes.c_int),
                                ("shortconv_backward_workspace_bytes", [d], i64),
                                ("shortconv_backward", [d] + [vp] * 11 + [i64, vp], ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _FN = lib
    return _FN


def shortconv_backward_workspace_bytes(B: int, T: int, C: int, K: int) -> int:
    """Workspace bytes of shortconv_backward for these sizes."""
    return M.size(_lib().shortconv_backward_workspace_bytes, ctypes.byref(ShortconvDesc(*M.sizes(B, T, C, K))))


def _act(act) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    return ACTS[act]


def _desc(x, y, B, T, C, K, act, S=0, lengths=None):
    M.sizes(B, T, C, K, S)
    return ShortconvDesc(B, T, C, K, M.dtype_code(x), M.dtype_code(y), _act(act), S, M.ptr(lengths))


def _inputs(x, w, bias, lengths, step):
    dev = M.gpu("x", x, 2 if step else 3)
    C = x.shape[-1]
    if w.dim() != 2 or w.shape[0] != C:
        raise ValueError(f"w must be [C, K] with C = {C}, got {tuple(w.shape)}")
    M.check("w", w, w.shape, torch.float32, dev)
    M.check_if("bias", bias, (C,), torch.float32, dev)
    M.check_if("lengths", lengths, (x.shape[0],), torch.int32, dev)
    return dev, x.shape[0], 1 if step else x.shape[1], C, w.shape[1]


def shortconv_forward(x, w, *, bias=None, state=None, lengths=None, act: str = "silu", y_dtype: Optional[str] = None,
                      y=None, state_out=None, return_state: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The convolution over T tokens after the inputs in `state` (None: zeros).  Returns (y,
    state_out); state_out is None when return_state is False and may be state (in place)."""
    dev, B, T, C, K = _inputs(x, w, bias, lengths, False)
    M.check_if("state", state, (B, K - 1, C), x.dtype, dev)
    y = M.output("y", y, x, y_dtype, dev)
    if state_out is not None:
        M.check("state_out", state_out, (B, K - 1, C), x.dtype, dev)
    elif return_state:
        state_out = torch.empty((B, max(K - 1, 0), C), dtype=x.dtype, device=dev)
    desc = _desc(x, y, B, T, C, K, act, 0, lengths)
    M.call(_lib().shortconv_forward, dev, ctypes.byref(desc), *M.ptrs(x, w, bias, state, y, state_out))
    return y, state_out


def shortconv_step(x, w, state, *, bias=None, state_index=None, act: str = "silu", y_dtype: Optional[str] = None,
                   y=None) -> torch.Tensor:
    """One token per row: x [B, C], state [S, K - 1, C] updated in place; returns y [B, C].
    state_index as in ssm.ssm_step."""
    dev, B, _, C, K = _inputs(x, w, bias, None, True)
    S = state.shape[0] if state.dim() else 0
    M.check("state", state, (S, K - 1, C), x.dtype, dev)
    M.check_if("state_index", state_index, (B,), torch.int32, dev)
    y = M.output("y", y, x, y_dtype, dev)
    desc = _desc(x, y, B, 1, C, K, act, S)
    M.call(_lib().shortconv_step, dev, ctypes.byref(desc), *M.ptrs(x, w, bias, state, state_index, y))
    return y


def shortconv_backward(x, w, dy, *, bias=None, state=None, dstate=None, lengths=None, act: str = "silu", workspace=None,
                       grads=None, return_dstate: bool = True) -> dict:
    """Gradients of <dy, y> + <dstate, state_out> for shortconv_forward with the same
    arguments.  dy of the y dtype, dstate [B, K - 1, C] float32 or None.  Returns a dict: x of
    x's dtype, w [C, K], bias [C] (None without bias), state [B, K - 1, C] float32 (None when
    return_dstate is False).  `grads` may supply output tensors under these keys (others: ValueError)."""
    dev, B, T, C, K = _inputs(x, w, bias, lengths, False)
    f32 = torch.float32
    M.check_if("state", state, (B, K - 1, C), x.dtype, dev)
    M.check("dy", dy, x.shape, dy.dtype, dev)
    M.check_if("dstate", dstate, (B, K - 1, C), f32, dev)
    out = M.gradients(grads, (("x", x, None, None), ("w", w, None, None), ("bias", bias, None, None),
                              ("state", x if return_dstate else None, (B, max(K - 1, 0), C), f32)), dev)
    desc = _desc(x, dy, B, T, C, K, act, 0, lengths)
    lib = _lib()
    need = M.size(lib.shortconv_backward_workspace_bytes, ctypes.byref(desc))
    ws, ws_bytes, keep = M.scratch(workspace, need, dev)
    M.call(lib.shortconv_backward, dev, ctypes.byref(desc),
           *M.ptrs(x, w, bias, state, dy, dstate, out["x"], out["w"], out["bias"], out["state"]), ws, ws_bytes)
    return out
