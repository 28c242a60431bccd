"""fp64 CPU oracle of linear attention with a decay for each head and of the layer
norm over a residual stream, with their gradients.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module.  It
shares no code with the HIP library.  Everything is evaluated as it is defined,
token by token and row by row (see include/linattn.h, include/layernorm.h).

`mag` and `grow` as in seq_oracle.py: with mag a function returns the same sums over
the absolute values of their terms; with grow = (g0, g1) every decay is
(1 + g0 + g1 |g|) times itself.

Pinned by tests/test_attn_oracle.py.
"""
from __future__ import annotations

import numpy as np

from .seq_oracle import _abs_if, _tokens, as_f64

__all__ = ["attn_forward", "attn_backward", "attn_step", "layer_forward", "layer_backward"]


def _parts(q, k, v, g, state, lengths):
    q, k, v, g, state = (as_f64(x) for x in (q, k, v, g, state))
    B, T = q.shape[:2]
    H = g.shape[-1]
    there, _ = _tokens(lengths, B, T)
    wide = lambda x: np.where(there[..., None, None], np.repeat(x, H // max(1, x.shape[2]), axis=2), 0.0)
    g = np.where(there[..., None], np.broadcast_to(g, (B, T, H)), 0.0)
    S = np.zeros((B, H, q.shape[3], v.shape[3])) if state is None else state
    return wide(q), wide(k), wide(v), g, S, there


def _decay(g, grow):
    with np.errstate(invalid="ignore"):
        return (np.exp(g) * np.where(np.isinf(g), 1.0, 1.0 + grow[0] + grow[1] * np.abs(g)))[..., None, None]


def attn_forward(q, k, v, g, scale=1.0, state=None, lengths=None, mag=False, grow=(0.0, 0.0)):
    """y [B, T, H, Dv], the last state [B, H, Dk, Dv], and the states before every token and behind the last."""
    q, k, v, g, S, _ = _parts(q, k, v, g, state, lengths)
    f = _abs_if(mag)
    B, T, H, _ = q.shape
    S = f(S)
    states, y = [S], np.zeros((B, T, H, v.shape[3]))
    for t in range(T):
        S = _decay(g[:, t], grow) * S + f(k[:, t])[..., None] * f(v[:, t])[..., None, :]
        states.append(S)
        y[:, t] = (f(q[:, t] * scale)[..., None] * S).sum(-2)
    return y, S, states


def attn_backward(q, k, v, g, dy, scale=1.0, state=None, dstate=None, lengths=None, mag=False, grow=(0.0, 0.0), sums=False):
    """A dict of the gradients of <dy, y> + <dstate, last state>.  sums: g's as the sum over all later
    tokens of <q, dq> and <k, dk> (with mag, of their absolute values), the way it is computed."""
    heads = [np.asarray(x).shape[2] for x in (q, k, v)]
    per_token = np.asarray(g).ndim == 3
    _, last, states = attn_forward(q, k, v, g, scale, state, lengths, mag, grow)
    q, k, v, g, S, there = _parts(q, k, v, g, state, lengths)
    f = _abs_if(mag)
    B, T, H, _ = q.shape
    dy = np.where(there[..., None, None], as_f64(dy), 0.0) * scale
    E = np.zeros_like(S) if dstate is None else f(as_f64(dstate))
    end = (E * last).sum((-1, -2))
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, T, H))
    for t in range(T - 1, -1, -1):
        E = E + f(q[:, t])[..., None] * f(dy[:, t])[..., None, :]
        dq[:, t] = (states[t + 1] * f(dy[:, t])[..., None, :]).sum(-1)
        dk[:, t] = (E * f(v[:, t])[..., None, :]).sum(-1)
        dv[:, t] = (E * f(k[:, t])[..., None]).sum(-2)
        a = _decay(g[:, t], grow)
        dg[:, t] = (a * E * states[t]).sum((-1, -2))
        E = a * E
    if sums:
        each = (f(q) * dq).sum(-1) + (1 if mag else -1) * (f(k) * dk).sum(-1)
        dg = np.cumsum(each[:, ::-1], 1)[:, ::-1] + end[:, None]
    dg = np.where(there[..., None], dg, 0.0)
    share = lambda d, n: np.where(there[..., None, None], d, 0.0).reshape(B, T, n, H // max(1, n), d.shape[3]).sum(3)
    return {"q": share(dq, heads[0]), "k": share(dk, heads[1]), "v": share(dv, heads[2]), "g": dg if per_token else dg.sum((0, 1)), "state": E}


def attn_step(q, k, v, g, state, index=None, scale=1.0, mag=False):
    """y [B, H, Dv] and the pool behind the step: the first row of those that name a state has it."""
    pool, B, H = as_f64(state).copy(), np.asarray(q).shape[0], np.asarray(g).shape[-1]
    f = _abs_if(mag)
    if mag:
        pool = np.abs(pool)
    y, taken = np.zeros((B, H, np.asarray(v).shape[2])), set()
    for b in range(B):
        s = b if index is None else int(index[b])
        if s < 0 or s >= len(pool) or s in taken:
            continue
        taken.add(s)
        one = lambda x: f(np.repeat(as_f64(x)[b], H // np.asarray(x).shape[1], axis=0))
        gb = as_f64(g)[b] if np.asarray(g).ndim == 2 else as_f64(g)
        pool[s] = np.exp(gb)[:, None, None] * pool[s] + one(k)[..., None] * one(v)[:, None, :]
        y[b] = (one(q)[..., None] * pool[s]).sum(1) * (abs(scale) if mag else scale)
    return y, pool


def layer_forward(h, weight=None, bias=None, eps=1e-5, lengths=None):
    """y, mean and rstd of the rows of h [B, T, C] (the stream as it is stored)."""
    h, weight, bias = (as_f64(x) for x in (h, weight, bias))
    B, T, C = h.shape
    there, _ = _tokens(lengths, B, T)
    h = np.where(there[..., None], h, 0.0)
    y, mean, rstd = np.zeros_like(h), np.zeros((B, T)), np.full((B, T), 1.0 / np.sqrt(eps))
    for b in range(B):
        for t in range(T):
            if there[b, t] and C:
                mean[b, t] = h[b, t].mean()
                rstd[b, t] = 1.0 / np.sqrt(((h[b, t] - mean[b, t]) ** 2).mean() + eps)
                y[b, t] = (h[b, t] - mean[b, t]) * rstd[b, t] * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    return y, mean, rstd


def layer_backward(h, dy, weight=None, dh=None, eps=1e-5, lengths=None, mag=False):
    """Gradients of <dy, y> + <dh, h>: of the stream, weight and bias."""
    f = _abs_if(mag)
    _, mean, rstd = layer_forward(h, weight, None, eps, lengths)
    h, dy, weight, dh = (as_f64(x) for x in (h, dy, weight, dh))
    there, _ = _tokens(lengths, *h.shape[:2])
    h, dy = np.where(there[..., None], h, 0.0), np.where(there[..., None], dy, 0.0)
    xh = f((h - mean[..., None]) * rstd[..., None])
    dxh = f(dy * (1.0 if weight is None else weight))
    sign = 1.0 if mag else -1.0
    C = max(1, h.shape[2])
    d = rstd[..., None] * (dxh + sign * dxh.sum(-1, keepdims=True) / C + sign * xh * (dxh * xh).sum(-1, keepdims=True) / C)
    d = d + (0.0 if dh is None else f(dh))
    return {"h": np.where(there[..., None], d, 0.0), "weight": (f(dy) * xh).sum((0, 1)), "bias": f(dy).sum((0, 1))}
