"""fp64 CPU oracle of the per-channel operators: the selective state space scan,
the short causal convolution and the group norm, with their gradients.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path imports this module.  It
shares no code with the HIP library.  Everything is evaluated as it is defined,
token by token (see include/ssm.h, include/shortconv.h, include/groupnorm.h).

Every function takes `mag`: with it, it returns, in place of its values, the same
sums over the absolute values of their terms.  A floating-point evaluation of a
sum is off by a small multiple of the rounding unit times that, which is what the
tests' tolerances are made of.  The scan's also take `grow` = (g0, g1): every decay
is then (1 + g0 + g1 |d A|) times itself, so that, with mag, the difference from
the result without it bounds what decays off by that much do to the result.

Pinned by tests/test_seq_oracle.py.
"""
from __future__ import annotations

import numpy as np

__all__ = ["as_f64", "sigmoid", "softplus", "scan_forward", "scan_backward", "conv_forward", "conv_backward",
           "norm_forward", "norm_backward"]


def as_f64(x):
    """Widen to float64; uint16 arrays are bf16 bit patterns."""
    if x is None:
        return None
    x = np.asarray(x)
    if x.dtype == np.uint16:
        return (x.astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)
    return x.astype(np.float64)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(x):
    return np.logaddexp(0.0, x)


def _dsilu(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def _abs_if(mag):
    return np.abs if mag else (lambda x: x)


def _tokens(lengths, B, T):
    """[B, T] truth values: the token belongs to its sequence."""
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths, dtype=np.int64), 0, T)
    return np.arange(T)[None] < n[:, None], n


def _scan_parts(x, dt, A, Bm, Cm, D, dt_bias, z, state, lengths, use_softplus):
    x, dt, A, Bm, Cm, D, dt_bias, z, state = (as_f64(v) for v in (x, dt, A, Bm, Cm, D, dt_bias, z, state))
    B, T, C = x.shape
    there, _ = _tokens(lengths, B, T)
    v = dt + (0.0 if dt_bias is None else dt_bias)
    d = softplus(v) if use_softplus else v
    d = np.where(there[..., None], d, 0.0)
    x = np.where(there[..., None], x, 0.0)
    rep = C // Bm.shape[2]
    Bc = np.where(there[..., None, None], np.repeat(Bm, rep, axis=2), 0.0)
    Cc = np.where(there[..., None, None], np.repeat(Cm, rep, axis=2), 0.0)
    z = None if z is None else np.where(there[..., None], z, 0.0)
    h0 = np.zeros((B, C, A.shape[1])) if state is None else state
    return x, v, d, A, Bc, Cc, (np.zeros(C) if D is None else D), z, h0, there


def _decay(dt_A, grow):
    return np.exp(dt_A) * (1.0 + grow[0] + grow[1] * np.abs(dt_A))


def scan_forward(x, dt, A, Bm, Cm, D=None, dt_bias=None, z=None, state=None, lengths=None, use_softplus=True, mag=False,
                 grow=(0.0, 0.0)):
    """y [B, T, C] and the final state [B, C, N]; also every state, [B, T + 1, C, N]."""
    x, v, d, A, Bc, Cc, D, z, h0, there = _scan_parts(x, dt, A, Bm, Cm, D, dt_bias, z, state, lengths, use_softplus)
    f = _abs_if(mag)
    B, T, C = x.shape
    hs = np.empty((B, T + 1) + h0.shape[1:])
    hs[:, 0] = f(h0)
    y = np.zeros((B, T, C))
    for t in range(T):
        hs[:, t + 1] = _decay(d[:, t, :, None] * A, grow) * hs[:, t] + f(d[:, t] * x[:, t])[..., None] * f(Bc[:, t])
        y[:, t] = (f(Cc[:, t]) * hs[:, t + 1]).sum(-1) + f(D * x[:, t])
    if z is not None:
        y = y * f(z * sigmoid(z))
    return np.where(there[..., None], y, 0.0), hs[:, T], hs


def scan_backward(x, dt, A, Bm, Cm, dy, D=None, dt_bias=None, z=None, state=None, dstate=None, lengths=None,
                  use_softplus=True, mag=False, grow=(0.0, 0.0)):
    """A dict of the gradients of <dy, y> + <dstate, final state>."""
    G = np.asarray(Bm).shape[2]
    _, _, hs = scan_forward(x, dt, A, Bm, Cm, D, dt_bias, z, state, lengths, use_softplus, mag, grow)
    x, v, d, A, Bc, Cc, D, z, h0, there = _scan_parts(x, dt, A, Bm, Cm, D, dt_bias, z, state, lengths, use_softplus)
    f = _abs_if(mag)
    B, T, C = x.shape
    N = A.shape[1]
    dy = np.where(there[..., None], as_f64(dy), 0.0)
    y0 = (f(Cc) * hs[:, 1:]).sum(-1) + f(D * x)
    dz = None if z is None else f(dy * _dsilu(z)) * y0
    do = f(dy) if z is None else f(dy * z * sigmoid(z))
    e = np.zeros((B, C, N)) if dstate is None else f(as_f64(dstate))
    dx, dd = np.zeros((B, T, C)), np.zeros((B, T, C))
    dB, dC = np.zeros((B, T, C, N)), np.zeros((B, T, C, N))
    dA = np.zeros((C, N))
    for t in range(T - 1, -1, -1):
        e = e + do[:, t, :, None] * f(Cc[:, t])
        a = _decay(d[:, t, :, None] * A, grow)
        dC[:, t] = do[:, t, :, None] * hs[:, t + 1]
        dB[:, t] = e * f(d[:, t] * x[:, t])[..., None]
        du = (e * f(Bc[:, t])).sum(-1)
        q = e * a * hs[:, t]
        dA += (q * f(d[:, t])[..., None]).sum(0)
        dd[:, t] = (q * f(A)).sum(-1) + du * f(x[:, t])
        dx[:, t] = du * f(d[:, t]) + do[:, t] * f(D)
        e = a * e
    sv = sigmoid(v) if use_softplus else np.ones_like(v)
    ddt = np.where(there[..., None], dd * sv, 0.0)
    g = {"x": dx, "dt": ddt, "z": dz, "A": dA, "B": dB.reshape(B, T, G, C // G, N).sum(3),
         "C": dC.reshape(B, T, G, C // G, N).sum(3), "D": (do * f(x)).sum((0, 1)), "dt_bias": ddt.sum((0, 1)), "state": e}
    return g


def _act(pre, silu):
    return pre * sigmoid(pre) if silu else pre


def conv_forward(x, w, bias=None, state=None, lengths=None, silu=True, mag=False):
    """y [B, T, C], the last K - 1 inputs [B, K - 1, C], the values before the activation."""
    x, w, bias, state = (as_f64(v) for v in (x, w, bias, state))
    f = _abs_if(mag)
    B, T, C = x.shape
    K = w.shape[1]
    there, n = _tokens(lengths, B, T)
    x = np.where(there[..., None], x, 0.0)
    before = np.zeros((B, K - 1, C)) if state is None else state
    xs = np.concatenate([before, x], 1)
    pre = np.zeros((B, T, C)) + (0.0 if bias is None else f(bias))
    for t in range(T):
        for k in range(K):
            pre[:, t] += f(xs[:, t + k] * w[:, k])
    out = np.stack([xs[b, n[b]:n[b] + K - 1] for b in range(B)]) if B else before
    y = pre if mag else _act(pre, silu)
    return np.where(there[..., None], y, 0.0), out, pre


def conv_backward(x, w, dy, bias=None, state=None, dstate=None, lengths=None, silu=True, mag=False):
    f = _abs_if(mag)
    _, _, pre = conv_forward(x, w, bias, state, lengths, silu)
    x, w, dy, state = (as_f64(v) for v in (x, w, dy, state))
    B, T, C = x.shape
    K = w.shape[1]
    there, n = _tokens(lengths, B, T)
    x, dy = np.where(there[..., None], x, 0.0), np.where(there[..., None], dy, 0.0)
    xs = np.concatenate([np.zeros((B, K - 1, C)) if state is None else state, x], 1)
    dpre = f(dy * (_dsilu(pre) if silu else 1.0))
    dxs = np.zeros_like(xs)
    dw = np.zeros((C, K))
    for t in range(T):
        for k in range(K):
            dxs[:, t + k] += dpre[:, t] * f(w[:, k])
            dw[:, k] += (dpre[:, t] * f(xs[:, t + k])).sum(0)
    if dstate is not None:
        for b in range(B):
            dxs[b, n[b]:n[b] + K - 1] += f(as_f64(dstate)[b])
    return {"x": dxs[:, K - 1:], "w": dw, "bias": dpre.sum((0, 1)), "state": dxs[:, :K - 1]}


def norm_forward(x, G, weight=None, bias=None, gate=None, silu=False, eps=1e-5, lengths=None):
    """y [B, T, C], mean and rstd [B, G]."""
    x, weight, bias, gate = (as_f64(v) for v in (x, weight, bias, gate))
    B, T, C = x.shape
    there, n = _tokens(lengths, B, T)
    y, mean, rstd = np.zeros((B, T, C)), np.zeros((B, G)), np.zeros((B, G))
    for b in range(B):
        for g in range(G):
            cs = slice(g * (C // G), (g + 1) * (C // G))
            v = x[b, :n[b], cs]
            m, var = (v.mean(), v.var()) if v.size else (0.0, 0.0)
            mean[b, g], rstd[b, g] = m, 1.0 / np.sqrt(var + eps)
            pre = (v - m) * rstd[b, g] * (1.0 if weight is None else weight[cs]) + (0.0 if bias is None else bias[cs])
            out = _act(pre, silu)
            y[b, :n[b], cs] = out if gate is None else out * gate[b, :n[b], cs]
    return y, mean, rstd


def norm_backward(x, G, dy, weight=None, bias=None, gate=None, silu=False, eps=1e-5, lengths=None, mag=False):
    """Gradients by the chain rule through the mean and the variance of each group."""
    f = _abs_if(mag)
    _, mean, rstd = norm_forward(x, G, weight, bias, gate, silu, eps, lengths)
    x, dy, weight, bias, gate = (as_f64(v) for v in (x, dy, weight, bias, gate))
    B, T, C = x.shape
    there, n = _tokens(lengths, B, T)
    w = np.ones(C) if weight is None else weight
    out = {"x": np.zeros((B, T, C)), "weight": np.zeros(C), "bias": np.zeros(C),
           "gate": None if gate is None else np.zeros((B, T, C))}
    for b in range(B):
        for g in range(G):
            cs = slice(g * (C // G), (g + 1) * (C // G))
            if n[b] == 0 or C == 0:
                continue
            xv, d = x[b, :n[b], cs], dy[b, :n[b], cs]
            xh = (xv - mean[b, g]) * rstd[b, g]
            pre = xh * w[cs] + (0.0 if bias is None else bias[cs])
            if gate is not None:
                out["gate"][b, :n[b], cs] = f(d * _act(pre, silu))
                d = d * gate[b, :n[b], cs]
            dpre = f(d * (_dsilu(pre) if silu else 1.0))
            out["weight"][cs] += (dpre * f(xh)).sum(0)
            out["bias"][cs] += dpre.sum(0)
            dxh = dpre * f(w[cs])
            # xh = (x - m) r, m = mean(x), r = (mean((x - m)^2) + eps)^(-1/2)
            minus = 1.0 if mag else -1.0
            out["x"][b, :n[b], cs] = rstd[b, g] * (dxh + minus * dxh.mean() + minus * f(xh) * (dxh * f(xh)).mean())
    return out
