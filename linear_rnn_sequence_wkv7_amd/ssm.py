"""Binding of the selective state space scan (include/ssm.h) on torch GPU tensors:
ssm_forward, ssm_step, ssm_backward.  Argument marshalling only; every step of the
computation runs in the library's HIP kernels, and without the library every call
raises.

    d_t = softplus(dt_t + dt_bias),  h_t = exp(d_t A) h_{t-1} + d_t x_t Bm_t,
    y_t = (Cm_t . h_t + D x_t) silu(z_t)

Shapes: x, dt, z, y [B, T, C]; Bm, Cm [B, T, G, N]; A [C, N] float32; D, dt_bias [C]
float32; states [B, C, N] float32; lengths [B] int32.  x, dt, z, Bm, Cm are all
float32 or all bfloat16; everything is contiguous and starts on 16 bytes (lengths and
state_index on 4).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _marshal as M
from .wkv7 import load_library

__all__ = ["ssm_forward", "ssm_step", "ssm_backward", "ssm_checkpoint_bytes", "ssm_backward_workspace_bytes",
           "CHECKPOINT_TOKENS", "SsmDesc", "EXPORTED_SYMBOLS"]

EXPORTED_SYMBOLS = ("ssm_checkpoint_bytes", "ssm_forward", "ssm_step", "ssm_backward_workspace_bytes", "ssm_backward")
CHECKPOINT_TOKENS = 32


class SsmDesc(ctypes.Structure):
    """Mirror of struct ssm_desc."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "N", "G", "in_dtype", "y_dtype", "dt_softplus", "S",
                                              "reserved")] + [("lengths", ctypes.c_void_p)]


_FN = None


def _lib():
    """The library with these functions' signatures declared (once)."""
    global _FN
    if _FN is None:
        lib = load_library()
        d, vp, i64 = ctypes.POINTER(SsmDesc), ctypes.c_void_p, ctypes.c_int64
        for name, args, res in (("ssm_checkpoint_bytes", [d], i64),
                                ("ssm_forward", [d] + [vp] * 13, ctypes.c_int),
                                ("ssm_step", [d] + [vp] * 12, ctypes.c_int),
                                ("ssm_backward_workspace_bytes", [d, ctypes.c_int], i64),
                                ("ssm_backward", [d] + [vp] * 22 + [i64, vp], ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _FN = lib
    return _FN


def _sizes(B, T, C, N, G=1, dtype=0):
    return SsmDesc(*M.sizes(B, T, C, N, G), in_dtype=dtype, y_dtype=dtype, dt_softplus=1)


def ssm_checkpoint_bytes(B: int, T: int, C: int, N: int) -> int:
    """Bytes of the states that ssm_forward can leave for ssm_backward."""
    return M.size(_lib().ssm_checkpoint_bytes, ctypes.byref(_sizes(B, T, C, N)))


def ssm_backward_workspace_bytes(B: int, T: int, C: int, N: int, *, G: int = 1, checkpoints: bool = True) -> int:
    """Workspace bytes of ssm_backward for these sizes, with or without checkpoints."""
    return M.size(_lib().ssm_backward_workspace_bytes, ctypes.byref(_sizes(B, T, C, N, G)), 0 if checkpoints else 1)


def _inputs(x, dt, A, Bm, Cm, D, dt_bias, z, lengths, step):
    """Check the inputs; the device and the sizes."""
    dev = M.gpu("x", x, 2 if step else 3)
    row, C = x.shape, x.shape[-1]
    f32 = torch.float32
    if A.dim() != 2 or A.shape[0] != C:
        raise ValueError(f"A must be [C, N] with C = {C}, got {tuple(A.shape)}")
    N = A.shape[1]
    if Bm.dim() != len(row) + 1:
        raise ValueError(f"Bm must be {'[B, G, N]' if step else '[B, T, G, N]'}, got {tuple(Bm.shape)}")
    G = Bm.shape[-2]
    if G == 0 or C % G:
        raise ValueError(f"{C} channels are not a multiple of G = {G}")
    dtype, vec, check = x.dtype, row[:-1] + (G, N), M.check
    check("A", A, (C, N), f32, dev)
    check("dt", dt, row, dtype, dev)
    check("Bm", Bm, vec, dtype, dev)
    check("Cm", Cm, vec, dtype, dev)
    if z is not None:
        check("z", z, row, dtype, dev)
    if D is not None:
        check("D", D, (C,), f32, dev)
    if dt_bias is not None:
        check("dt_bias", dt_bias, (C,), f32, dev)
    if lengths is not None:
        check("lengths", lengths, (row[0],), torch.int32, dev)
    return dev, row[0], 1 if step else row[1], C, N, G


def _desc(x, y, B, T, C, N, G, softplus, lengths=None, S=0):
    M.sizes(B, T, C, N, G, S)
    return SsmDesc(B, T, C, N, G, M.dtype_code(x), M.dtype_code(y), 1 if softplus else 0, S, 0, M.ptr(lengths))


def _check_checkpoints(checkpoints, B, T, C, N, dev):
    if checkpoints is None:
        return
    need = B * ((T + CHECKPOINT_TOKENS - 1) // CHECKPOINT_TOKENS) * C * N * 4
    if checkpoints.device != dev or not checkpoints.is_contiguous() or checkpoints.numel() * checkpoints.element_size() < need:
        raise ValueError(f"checkpoints must be a contiguous tensor of at least {need} bytes on {dev}")


def ssm_forward(x, dt, A, Bm, Cm, *, D=None, dt_bias=None, z=None, state=None, lengths=None, softplus: bool = True,
                y_dtype: Optional[str] = None, y=None, state_out=None, return_state: bool = True,
                checkpoints=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The scan over T tokens from `state` (None: zeros).  Returns (y, state_out); outputs
    are allocated unless given (state_out may be state: in place), state_out is None when
    return_state is False.  lengths: tokens of each sequence (the others are padding: y 0,
    state untouched).  checkpoints: a buffer of ssm_checkpoint_bytes(B, T, C, N) bytes that
    the call fills for ssm_backward."""
    dev, B, T, C, N, G = _inputs(x, dt, A, Bm, Cm, D, dt_bias, z, lengths, False)
    M.check_if("state", state, (B, C, N), torch.float32, dev)
    y = M.output("y", y, x, y_dtype, dev)
    if state_out is not None:
        M.check("state_out", state_out, (B, C, N), torch.float32, dev)
    elif return_state:
        state_out = torch.empty((B, C, N), dtype=torch.float32, device=dev)
    _check_checkpoints(checkpoints, B, T, C, N, dev)
    desc = _desc(x, y, B, T, C, N, G, softplus, lengths)
    M.call(_lib().ssm_forward, dev, ctypes.byref(desc),
           *M.ptrs(x, dt, A, Bm, Cm, D, dt_bias, z, state, y, state_out, checkpoints))
    return y, state_out


def ssm_step(x, dt, A, Bm, Cm, state, *, D=None, dt_bias=None, z=None, state_index=None, softplus: bool = True,
             y_dtype: Optional[str] = None, y=None) -> torch.Tensor:
    """One token per row: x, dt, z [B, C], Bm, Cm [B, G, N], state [S, C, N] updated in place;
    returns y [B, C].  Row b works on state state_index[b] (int32 [B]; None: state b).  A row
    whose index is outside 0 .. S - 1, or that an earlier row already names, has no request:
    its y is 0 and no state changes for it."""
    dev, B, _, C, N, G = _inputs(x, dt, A, Bm, Cm, D, dt_bias, z, None, True)
    S = state.shape[0] if state.dim() else 0
    M.check("state", state, (S, C, N), torch.float32, dev)
    M.check_if("state_index", state_index, (B,), torch.int32, dev)
    y = M.output("y", y, x, y_dtype, dev)
    desc = _desc(x, y, B, 1, C, N, G, softplus, None, S)
    M.call(_lib().ssm_step, dev, ctypes.byref(desc), *M.ptrs(x, dt, A, Bm, Cm, D, dt_bias, z, state, state_index, y))
    return y


def ssm_backward(x, dt, A, Bm, Cm, dy, *, D=None, dt_bias=None, z=None, state=None, dstate=None, lengths=None,
                 softplus: bool = True, checkpoints=None, workspace=None, grads=None, return_dstate: bool = True) -> dict:
    """Gradients of <dy, y> + <dstate, state_out> for ssm_forward with the same arguments.

    dy [B, T, C] of the y dtype; dstate [B, C, N] float32 or None; checkpoints as ssm_forward
    filled them (None: the states are computed again, into the workspace).  Returns a dict:
    x, dt, z, B, C of the input dtype, A [C, N], D, dt_bias [C], state [B, C, N] float32 (z, D
    and dt_bias None where they are not inputs, state None when return_dstate is False).
    `grads` may supply output tensors under these keys (others: ValueError)."""
    dev, B, T, C, N, G = _inputs(x, dt, A, Bm, Cm, D, dt_bias, z, lengths, False)
    f32 = torch.float32
    M.check_if("state", state, (B, C, N), f32, dev)
    M.check("dy", dy, x.shape, dy.dtype, dev)
    M.check_if("dstate", dstate, (B, C, N), f32, dev)
    _check_checkpoints(checkpoints, B, T, C, N, dev)
    out = M.gradients(grads, (("x", x, None, None), ("dt", dt, None, None), ("z", z, None, None), ("B", Bm, None, None),
                              ("C", Cm, None, None), ("A", A, None, None), ("D", D, None, None), ("dt_bias", dt_bias, None, None),
                              ("state", x if return_dstate else None, (B, C, N), f32)), dev)
    desc = _desc(x, dy, B, T, C, N, G, softplus, lengths)
    lib = _lib()
    need = M.size(lib.ssm_backward_workspace_bytes, ctypes.byref(desc), 1 if checkpoints is None else 0)
    ws, ws_bytes, keep = M.scratch(workspace, need, dev)
    M.call(lib.ssm_backward, dev, ctypes.byref(desc),
           *M.ptrs(x, dt, A, Bm, Cm, D, dt_bias, z, state, dy, dstate, checkpoints, out["x"], out["dt"], out["A"], out["B"], out["C"],
                   out["D"], out["dt_bias"], out["z"], out["state"]), ws, ws_bytes)
    return out
