"""Inputs and error bounds of linear attention's and the layer norm's GPU tests (see seq_util.py)."""
import numpy as np

from oracle import attn_oracle as O
from tests.seq_util import U, as_dtype


def attn_inputs(seed, B, T, H, Dk, Dv, Hq=0, Hk=0, Hv=0, dtype="f32", per_token=True, state=False, step=False, rate=0.3):
    rng = np.random.default_rng(seed)
    row = (B,) if step else (B, T)
    r = lambda *s: rng.standard_normal(s)
    return {"q": as_dtype(r(*row, Hq or H, Dk), dtype), "k": as_dtype(r(*row, Hk or H, Dk), dtype), "v": as_dtype(r(*row, Hv or H, Dv), dtype),
            "g": (-rate * np.exp(r(*(row if per_token else ()), H))).astype(np.float32),
            "state": r(B, H, Dk, Dv).astype(np.float32) if state else None}


def _grown(f, T):
    """Values, sums of magnitudes, and those with every decay off by what it may be: exp(X_t - X_i) is an
    exponential (2 U) of a difference good to U, and there are at most one for each chunk and two more."""
    return f(), f(mag=True), f(mag=True, grow=(3 * U, 3 * U))


def attn_bounds(x, scale, lengths=None):
    """Reference values and error bounds of y and the last state.  A sum is off by 2 U of its terms'
    magnitudes for each addition in a row (matrix cores): Dk products twice, 64 tokens and the tokens of the
    state, 250 for all single operations.  Of bf16 operands y's state and P are sums of two bf16: 2^-17 each."""
    T, Dk = np.asarray(x["q"]).shape[1], np.asarray(x["q"]).shape[3]
    split = 2.0 ** -16 if np.asarray(x["q"]).dtype == np.uint16 else 0.0
    f = lambda **kw: O.attn_forward(x["q"], x["k"], x["v"], x["g"], scale, x["state"], lengths, **kw)[:2]
    ref, m, w = _grown(f, T)
    rest = (2 * (2 * Dk + T) + 250) * U
    return ref, (w[0] - m[0] + (rest + split) * w[0], w[1] - m[1] + (2 * T + 250) * U * w[1])


def attn_grad_bounds(x, dy, dstate, scale, lengths=None):
    """The same of the gradients, whose operands are whole (three bf16).  g's is a difference of sums over
    all later tokens: its bound is that of their magnitudes."""
    T, D = np.asarray(x["q"]).shape[1], max(np.asarray(x["q"]).shape[3], np.asarray(x["v"]).shape[3])
    H = np.asarray(x["g"]).shape[-1]
    f = lambda **kw: O.attn_backward(x["q"], x["k"], x["v"], x["g"], dy, scale, x["state"], dstate, lengths, sums=bool(kw), **kw)
    ref, m, w = _grown(f, T)
    rest = (2 * (3 * D + T) + 250 + H) * U
    return ref, {n: w[n] - m[n] + rest * w[n] for n in ref}


def norm_inputs(seed, B, T, C, x_dtype, h_dtype, residual=True):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)
    return {"x": as_dtype(r(B, T, C) * 0.7 + 0.1, x_dtype if residual else h_dtype), "residual": as_dtype(r(B, T, C) * 1.5, h_dtype) if residual else None,
            "weight": (1 + 0.2 * r(C)).astype(np.float32), "bias": (0.2 * r(C)).astype(np.float32)}


def stream(x):
    """h as it is stored: the fp32 sum, rounded to the stream's type."""
    from oracle.seq_oracle import as_f64
    if x["residual"] is None:
        return x["x"]
    total = (as_f64(x["x"]) + as_f64(x["residual"])).astype(np.float32)
    return as_dtype(total, "bf16" if x["residual"].dtype == np.uint16 else "f32")


def norm_bounds(h, weight, bias, eps, lengths=None):
    """y, mean and rstd.  A sum over C channels: runs of 16 in a lane, then a tree over the row's waves, or runs
    of C / 1024: 60 + C / 1024 units of the largest |h| in the mean, as much relative in the variance (of
    differences that are off by the mean's error), half in rstd."""
    (y, mean, rstd), C = O.layer_forward(h, weight, bias, eps, lengths), np.asarray(h).shape[2]
    from oracle.seq_oracle import _tokens, as_f64
    there, _ = _tokens(lengths, *y.shape[:2])
    top = np.max(np.abs(np.where(there[..., None], as_f64(h), 0.0)), -1, initial=0.0)
    n = (60 + C / 1024) * U
    m_tol = n * top
    # d var <= 2 |d| e + e^2 + n var, with the mean's own error second order; rstd' = rstd^3 / 2
    r_tol = rstd * (2 * n + 2 * (m_tol * rstd) ** 2)
    xh = np.abs((np.where(there[..., None], as_f64(h), 0.0) - mean[..., None]) * rstd[..., None])
    xh_tol = (m_tol * rstd)[..., None] + xh * ((r_tol / rstd)[..., None] + 4 * U)
    w = 1.0 if weight is None else np.abs(weight)
    y_tol = w * xh_tol + 4 * U * (w * xh + (0.0 if bias is None else np.abs(bias)))
    return (y, mean, rstd), (y_tol, m_tol, r_tol), xh_tol


def norm_grad_bounds(h, dy, weight, dh, eps, lengths=None):
    ref = O.layer_backward(h, dy, weight, dh, eps, lengths)
    mag = O.layer_backward(h, dy, weight, dh, eps, lengths, mag=True)
    _, (_, _, _), xh_tol = norm_bounds(h, weight, None, eps, lengths)
    from oracle.seq_oracle import _tokens, as_f64
    rows, C = np.asarray(h).shape[0] * np.asarray(h).shape[1], max(1, np.asarray(h).shape[2])
    there, _ = _tokens(lengths, *np.asarray(h).shape[:2])
    d = np.where(there[..., None], np.abs(as_f64(dy)), 0.0)
    dxh = d * (1.0 if weight is None else np.abs(weight))
    (_, _, rstd), _, _ = norm_bounds(h, weight, None, eps, lengths)
    xh = np.abs((np.where(there[..., None], as_f64(h), 0.0) - O.layer_forward(h, None, None, eps, lengths)[1][..., None]) * rstd[..., None])
    # xh's error passes through: its own factor, and the mean of dxh xh; rstd's through all
    through = rstd[..., None] * (xh_tol * np.mean(dxh * xh, -1, keepdims=True) + xh * np.mean(dxh * xh_tol, -1, keepdims=True)) if C else 0.0
    n = (120 + C / 512) * U
    sums = (60 + rows / 8) * U
    return ref, {"h": np.where(there[..., None], through + n * mag["h"], 0.0), "weight": (d * xh_tol).sum((0, 1)) + sums * mag["weight"], "bias": sums * mag["bias"]}
