"""Binding of the layer norm with the residual stream's sum in front of it
(include/layernorm.h) on torch GPU tensors: layernorm_forward, layernorm_backward.
Argument marshalling only; without the library every call raises.

    h = x + residual,  y = (h - mean) rstd weight + bias      per row of C channels

Shapes: x, residual, h, y [B, T, C]; weight, bias [C] float32; mean, rstd [B, T] float32;
lengths [B] int32.  residual and h have the stream's type, which may be another than x's.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _marshal as M
from .wkv7 import load_library

__all__ = ["layernorm_forward", "layernorm_backward", "layernorm_backward_workspace_bytes", "LayernormDesc", "EXPORTED_SYMBOLS"]

EXPORTED_SYMBOLS = ("layernorm_forward", "layernorm_backward_workspace_bytes", "layernorm_backward")


class LayernormDesc(ctypes.Structure):
    """Mirror of struct layernorm_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "x_dtype", "h_dtype", "y_dtype")] + \
               [("eps", ctypes.c_float), ("reserved", ctypes.c_int32), ("lengths", ctypes.c_void_p)]


_FN = None


def _lib():
    """The library with these functions' signatures declared (once)."""
    global _FN
    if _FN is None:
        lib = load_library()
        d, vp, i64 = ctypes.POINTER(LayernormDesc), ctypes.c_void_p, ctypes.c_int64
        for name, args, res in (("layernorm_forward", [d] + [vp] * 9, ctypes.c_int),
                                ("layernorm_backward_workspace_bytes", [d], i64),
                                ("layernorm_backward", [d] + [vp] * 12 + [i64, vp], ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _FN = lib
    return _FN


def layernorm_backward_workspace_bytes(B: int, T: int, C: int) -> int:
    """Workspace bytes of layernorm_backward for these sizes, of any types."""
    return max(M.size(_lib().layernorm_backward_workspace_bytes, ctypes.byref(LayernormDesc(*M.sizes(B, T, C), d, d, d, 1.0))) for d in (0, 1))


def _inputs(name, x, weight, bias, lengths):
    dev = M.gpu(name, x, 3)
    B, T, C = x.shape
    M.check_if("weight", weight, (C,), torch.float32, dev)
    M.check_if("bias", bias, (C,), torch.float32, dev)
    M.check_if("lengths", lengths, (B,), torch.int32, dev)
    return dev, B, T, C


def _desc(B, T, C, x, h, y, eps, lengths):
    M.sizes(B, T, C)
    return LayernormDesc(B, T, C, M.dtype_code(x), M.dtype_code(h), M.dtype_code(y), eps, 0, M.ptr(lengths))


def layernorm_forward(x, *, residual=None, weight=None, bias=None, eps: float = 1e-5, lengths=None, y_dtype: Optional[str] = None, y=None,
                      h=None, mean=None, rstd=None, return_stats: bool = True
                      ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Returns (y, h, mean, rstd).  h = x + residual in residual's type (h may be given as residual
    itself: the stream moves on in place); without a residual it is x.  mean and rstd, which
    layernorm_backward takes, are None when return_stats is False and they are not given."""
    dev, B, T, C = _inputs("x", x, weight, bias, lengths)
    y = M.output("y", y, x, y_dtype, dev)
    if residual is None:
        if h is not None:
            raise ValueError("h is given but residual is None")
        stream = x
    else:
        M.check("residual", residual, x.shape, residual.dtype, dev)
        h = torch.empty_like(residual) if h is None else h
        M.check("h", h, x.shape, residual.dtype, dev)
        stream = h
    if return_stats:
        mean = torch.empty((B, T), dtype=torch.float32, device=dev) if mean is None else mean
        rstd = torch.empty((B, T), dtype=torch.float32, device=dev) if rstd is None else rstd
    M.check_if("mean", mean, (B, T), torch.float32, dev)
    M.check_if("rstd", rstd, (B, T), torch.float32, dev)
    desc = _desc(B, T, C, x, stream, y, eps, lengths)
    M.call(_lib().layernorm_forward, dev, ctypes.byref(desc), *M.ptrs(x, residual, weight, bias, h, y, mean, rstd))
    return y, stream, mean, rstd


def layernorm_backward(h, dy, mean, rstd, *, weight=None, bias=None, dh=None, lengths=None, x_dtype: Optional[str] = None, workspace=None,
                       grads=None) -> dict:
    """Gradients of <dy, y> + <dh, h> for layernorm_forward; h, mean and rstd as it returned them.

    Returns a dict: h, of h's type, the gradient of the stream and so of the residual; x, the same
    of x_dtype ("f32" or "bf16"; None: of h's type, and then it is h's tensor); weight and bias
    [C] float32 (None where they are not inputs).  `grads` may supply output tensors under these
    keys (others: ValueError); grads["h"] may be dh."""
    dev, B, T, C = _inputs("h", h, weight, bias, lengths)
    f32 = torch.float32
    M.check("dy", dy, h.shape, dy.dtype, dev)
    M.check_if("dh", dh, h.shape, h.dtype, dev)
    M.check("mean", mean, (B, T), f32, dev)
    M.check("rstd", rstd, (B, T), f32, dev)
    other = M.dtype_named(x_dtype, h.dtype)
    apart = other != h.dtype or bool(grads and grads.get("x") is not None)
    out = M.gradients(grads, (("h", h, None, None), ("x", h if apart else None, h.shape, other), ("weight", weight, None, None),
                              ("bias", bias, None, None)), dev)
    desc = LayernormDesc(*M.sizes(B, T, C), M.dtype_code(out["x"] if apart else h), M.dtype_code(h), M.dtype_code(dy), 1.0, 0, M.ptr(lengths))
    lib = _lib()
    ws, ws_bytes, keep = M.scratch(workspace, M.size(lib.layernorm_backward_workspace_bytes, ctypes.byref(desc)), dev)
    M.call(lib.layernorm_backward, dev, ctypes.byref(desc),
           *M.ptrs(h, weight, bias, dy, dh, mean, rstd, out["h"], out["x"], out["weight"], out["bias"]), ws, ws_bytes)
    if not apart:
        out["x"] = out["h"]
    return out
