"""Inputs, tolerances and comparisons of the per-channel operators' GPU tests.

Tolerances are error bounds worked out before any run.  U is the rounding unit of
fp32 (a rounding is off by at most U relative to the value), exponentials,
logarithms and reciprocals of the hardware are good to one unit in the last place
(2 U).  A result rounded to bf16 is off by 2^-8 more, relative to it.
"""
import numpy as np

from linear_rnn_sequence_wkv7_amd import inputs as G
from oracle import seq_oracle as O

U = 2.0 ** -24
BF16 = 2.0 ** -8


def as_dtype(x, dtype):
    """fp64 values -> fp32, or bf16 bit patterns."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    return x if dtype == "f32" else G.f32_to_bf16_bits(x)


def check(what, got, ref, tol, bf16=False):
    """|got - ref| <= tol (an array or a number), plus the rounding of a bf16 result."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    if ref.size == 0:
        return
    assert np.all(np.isfinite(got)), f"{what}: {np.sum(~np.isfinite(got))} values are not finite"
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), ref.shape)
    allow = tol + (BF16 * (np.abs(ref) + tol) if bf16 else 0.0) + 1e-37
    off = np.abs(got - ref)
    at = np.unravel_index(np.argmax(off / allow), ref.shape)
    assert off[at] <= allow[at], f"{what} at {at}: got {got[at]:.9g}, expected {ref[at]:.9g}, off {off[at]:.3g}, allowed {allow[at]:.3g}"


def scan_inputs(seed, B, T, C, N, G_=1, dtype="f32", z=True, D=True, bias=True, state=False, step=False):
    rng = np.random.default_rng(seed)
    row = (B, C) if step else (B, T, C)
    r = lambda *s, std=1.0: rng.standard_normal(s) * std
    x = {"x": as_dtype(r(*row), dtype), "dt": as_dtype(r(*row, std=0.7), dtype),
         "A": (-np.exp(rng.uniform(-3, 1.2, (C, N)))).astype(np.float32),
         "Bm": as_dtype(r(*row[:-1], G_, N), dtype), "Cm": as_dtype(r(*row[:-1], G_, N), dtype),
         "D": r(C).astype(np.float32) if D else None,
         "dt_bias": (r(C, std=0.5) - 1.0).astype(np.float32) if bias else None,
         "z": as_dtype(r(*row), dtype) if z else None,
         "state": r(B, C, N).astype(np.float32) if state else None}
    return x


def scan_bounds(x, T, lengths, softplus, dy=None, dstate=None, B=1, Cg=1):
    """Reference values and error bounds of the scan (of its gradients with dy).

    A decay exp2(d (A log2 e)): the exponent's three roundings and d's own error (softplus: an
    exponential, the logarithm's series and its division, 24 + 4 |v| units at the most) count
    times |d A|; the exponential and the products with the decay are 8 units.  All the other
    operations of a term and of its sum are counted together: 80, the N states, a tree over the
    16 channels of a wave, the blocks of channels, the rounds of 16 tokens, the batch."""
    v = O.as_f64(x["dt"]) + (0 if x["dt_bias"] is None else x["dt_bias"])
    vmax = float(np.max(np.abs(v[np.isfinite(v)]))) if v.size else 0.0
    zmax = 0.0 if x["z"] is None or np.size(x["z"]) == 0 else float(np.nanmax(np.abs(np.where(np.isfinite(O.as_f64(x["z"])), O.as_f64(x["z"]), 0))))
    d_err = 24 + 4 * vmax
    grow = (8 * U, (4 + d_err) * U)
    rest = (80 + x["A"].shape[1] + Cg / 4 + T / 8 + B + 2 * d_err + 4 * zmax) * U
    kw = dict(D=x["D"], dt_bias=x["dt_bias"], z=x["z"], state=x["state"], lengths=lengths, use_softplus=softplus)
    args = (x["x"], x["dt"], x["A"], x["Bm"], x["Cm"])
    if dy is None:
        ref = O.scan_forward(*args, **kw)[:2]
        m, g = O.scan_forward(*args, **kw, mag=True)[:2], O.scan_forward(*args, **kw, mag=True, grow=grow)[:2]
        return ref, [gi - mi + rest * gi for mi, gi in zip(m, g)]
    ref = O.scan_backward(*args, dy, **kw, dstate=dstate)
    m = O.scan_backward(*args, dy, **kw, dstate=dstate, mag=True)
    g = O.scan_backward(*args, dy, **kw, dstate=dstate, mag=True, grow=grow)
    # dz's factor silu' has a sum of both signs in it: sigmoid (1 + z (1 - sigmoid)), at most 1 + |z| before it is small
    tol = {k: None if ref[k] is None else g[k] - m[k] + rest * g[k] for k in ref}
    if ref["z"] is not None:
        y0 = O.scan_forward(*args, **{**kw, "z": None}, mag=True, grow=grow)[0]
        y1 = O.scan_forward(*args, **{**kw, "z": None}, mag=True)[0]
        tol["z"] = np.abs(O.as_f64(dy)) * (1.1 * (y0 - y1) + (rest + 16 * (1 + zmax) * U) * y0)
    return ref, tol


def conv_bounds(x, w, bias, state, lengths, silu, dy=None, dstate=None):
    """Reference values and error bounds of the convolution.

    The value before the activation: K + 2 operations.  SiLU passes an error on with a slope of at
    most 1.1 and adds its own, 6 + 2 |pre| units of its result; SiLU' has a slope of at most 0.5 and is
    off by up to 20 (1 + |pre|) units itself.  Sums over T tokens and the batch: runs of at most 32
    tokens, then a tree."""
    K = w.shape[1]
    ref_y, ref_s, pre = O.conv_forward(x, w, bias, state, lengths, silu)
    mag, _, _ = O.conv_forward(x, w, bias, state, lengths, silu, mag=True)
    if dy is None:
        return (ref_y, ref_s), (1.1 * (K + 2) * U * mag + (6 + 2 * np.abs(np.where(ref_y != 0, pre, 0))) * U * np.abs(ref_y), 0.0)
    ref = O.conv_backward(x, w, dy, bias, state, dstate, lengths, silu)
    plain = O.conv_backward(x, w, dy, bias, state, dstate, lengths, False, mag=True)   # with |dy| for |dpre|
    T, B = ref_y.shape[1], ref_y.shape[0]
    top = float(np.max(mag)) if mag.size else 0.0
    kappa = 0.5 * (K + 2) * top + 20 * (1 + top) if silu else 0.0
    return ref, {k: (kappa + 1.1 * (K + 40 + T / 8 + B)) * U * plain[k] for k in plain}


def norm_bounds(x, G_, weight, bias, gate, silu, eps, lengths, dy=None):
    """Reference values and error bounds of the group norm, from the largest values involved.

    A mean and a variance are trees over at most 64 positions and the lanes and blocks joined: 60
    units of the largest |x| in the mean, and so in x - mean; that times rstd is xh's error E.  Then
    as in conv_bounds, with the two means that dx takes off."""
    xf, w = O.as_f64(x), np.ones(1) if weight is None else weight
    ref, mean, rstd = O.norm_forward(x, G_, weight, bias, gate, silu, eps, lengths)
    top = lambda a: float(np.max(np.abs(a))) if a is not None and np.size(a) else 0.0
    there, _ = O._tokens(lengths, xf.shape[0], xf.shape[1])
    xf = np.where(there[..., None], xf, 0.0)
    rm, xm, wm, bm = top(rstd), top(xf), top(w), top(bias)
    gm = 1.0 if gate is None else top(np.where(there[..., None], O.as_f64(gate), 0.0))
    xhm = min(2 * xm * rm, np.sqrt(max(1, xf[0].size if xf.size else 1)))
    E = 60 * U * rm * xm + 60 * U * xhm
    pm = xhm * wm + bm
    e_pre = wm * E + 4 * U * pm
    e_act = 1.1 * e_pre + (10 + 2 * pm) * U * pm if silu else e_pre
    if dy is None:
        return (ref, mean, rstd), (e_act * gm + 4 * U * pm * gm, 60 * U * xm, 60 * U * rm + 120 * U * rm * rm * xm * min(xhm, 4.0))
    g = O.norm_backward(x, G_, dy, weight, bias, gate, silu, eps, lengths)
    mag = O.norm_backward(x, G_, dy, weight, bias, gate, silu, eps, lengths, mag=True)
    dm = top(np.where(there[..., None], O.as_f64(dy), 0.0))
    e_d = dm * gm * (0.5 * e_pre + 20 * (1 + pm) * U if silu else 4 * U)
    n = int(there.sum())
    slope = 1.1 if silu else 1.0
    tol = {"x": rm * (wm * e_d * (2 + xhm) + 2 * slope * wm * dm * gm * (1 + xhm) * E) + 200 * U * mag["x"],
           "weight": n * (e_d * xhm + slope * dm * gm * E) + (60 + n / 8) * U * mag["weight"],
           "bias": n * e_d + (60 + n / 8) * U * mag["bias"],
           "gate": None if gate is None else dm * e_act + 4 * U * dm * pm}
    return g, tol
