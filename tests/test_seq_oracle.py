"""Pins of oracle/seq_oracle.py (CPU): hand-worked values, closed forms, and every
gradient against central differences of the forward."""
import numpy as np
import pytest

from oracle import seq_oracle as O


def _close(a, b, tol):
    a, b = np.asarray(a, float), np.asarray(b, float)
    assert a.shape == b.shape
    if a.size:
        assert np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b)))


def test_scan_by_hand():
    """One channel, two states, two tokens with d = 1 and 2 (no softplus)."""
    x, dt = np.array([[[2.0], [3.0]]]), np.array([[[1.0], [2.0]]])
    A = np.array([[-np.log(2.0), 0.0]])
    Bm, Cm = np.array([[[[1.0, -1.0]], [[0.5, 2.0]]]]), np.array([[[[1.0, 10.0]], [[2.0, 1.0]]]])
    h0 = np.array([[[4.0, 1.0]]])
    # h_1 = (0.5 * 4 + 2, 1 - 2) = (4, -1); h_2 = (0.25 * 4 + 6 * 0.5, -1 + 6 * 2) = (4, 11)
    y, h, _ = O.scan_forward(x, dt, A, Bm, Cm, D=np.array([0.5]), state=h0, use_softplus=False)
    _close(h, [[[4.0, 11.0]]], 1e-14)
    _close(y, [[[4.0 - 10.0 + 1.0], [8.0 + 11.0 + 1.5]]], 1e-14)


def test_scan_limits():
    rng = np.random.default_rng(0)
    B, T, C, N = 2, 6, 3, 4
    x, dt = rng.standard_normal((B, T, C)), rng.standard_normal((B, T, C))
    Bm, Cm = rng.standard_normal((B, T, 1, N)), rng.standard_normal((B, T, 1, N))
    d = O.softplus(dt)
    # no decay: a running sum
    y, h, _ = O.scan_forward(x, dt, np.zeros((C, N)), Bm, Cm)
    run = np.cumsum((d * x)[..., None] * Bm, axis=1)
    _close(h, run[:, -1], 1e-13)
    _close(y, (Cm * run).sum(-1), 1e-13)
    # total decay: only the token itself
    y, _, _ = O.scan_forward(x, dt, np.full((C, N), -1e9), Bm, Cm, state=rng.standard_normal((B, C, N)))
    _close(y, d * x * (Bm * Cm).sum(-1), 1e-13)
    # a padded token is as if it were not there, whatever it holds
    x2, dt2 = x.copy(), dt.copy()
    x2[1, 4:], dt2[1, 4:] = np.nan, np.inf
    A = -np.exp(rng.standard_normal((C, N)))
    y, h, _ = O.scan_forward(x2, dt2, A, Bm, Cm, lengths=[6, 4])
    y4, h4, _ = O.scan_forward(x[:, :4], dt[:, :4], A, Bm[:, :4], Cm[:, :4])
    _close(y[1, :4], y4[1], 1e-14)
    _close(h[1], h4[1], 1e-14)
    assert np.all(y[1, 4:] == 0)


def test_conv_by_hand_and_against_numpy():
    x = np.array([[[1.0], [2.0], [3.0]]])
    y, s, _ = O.conv_forward(x, np.array([[10.0, 1.0]]), np.array([0.5]), np.array([[[7.0]]]), silu=False)
    _close(y, [[[70 + 1.5], [10 + 2.5], [20 + 3.5]]], 1e-14)
    _close(s, [[[3.0]]], 0)
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((1, 20, 1)), rng.standard_normal((1, 4))
    y, _, _ = O.conv_forward(x, w, silu=False)
    _close(y[0, :, 0], np.convolve(x[0, :, 0], w[0, ::-1])[:20], 1e-13)
    # a sequence of one token keeps the younger inputs of its state
    st = rng.standard_normal((1, 3, 1))
    _, s, _ = O.conv_forward(x, w, state=st, lengths=[1])
    _close(s[0, :, 0], [st[0, 1, 0], st[0, 2, 0], x[0, 0, 0]], 0)


def test_norm_definition():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 5, 6)) * 3 + 1
    y, mean, rstd = O.norm_forward(x, 2, eps=1e-12)
    g = y.reshape(2, 5, 2, 3)
    _close(g.mean((1, 3)), np.zeros((2, 2)), 1e-12)
    _close(g.var((1, 3)), np.ones((2, 2)), 1e-9)
    y, mean, rstd = O.norm_forward(x, 2, lengths=[5, 0], eps=0.25)
    assert np.all(y[1] == 0) and np.all(mean[1] == 0) and np.all(rstd[1] == 2.0)


def _check_gradients(loss, args, grads, names):
    """Central differences of loss(**args) in every entry of the named arrays."""
    h = 1e-6
    for n in names:
        a, num = args[n], np.zeros(args[n].shape)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = loss(**args)
            a[i] = keep - h
            num[i] = (up - loss(**args)) / (2 * h)
            a[i] = keep
        _close(grads[n], num, 5e-8)


@pytest.mark.parametrize("lengths", [None, [4, 0, 2]])
@pytest.mark.parametrize("gated", [False, True])
def test_scan_gradients(lengths, gated):
    rng = np.random.default_rng(3)
    B, T, C, N, G = 3, 4, 4, 3, 2
    r = lambda *s: rng.standard_normal(s)
    args = dict(x=r(B, T, C), dt=r(B, T, C), A=-np.exp(r(C, N)), B=r(B, T, G, N), C=r(B, T, G, N), D=r(C), dt_bias=r(C),
                state=r(B, C, N))
    if gated:
        args["z"] = r(B, T, C)
    dy, ds = r(B, T, C), r(B, C, N)

    def loss(x, dt, A, B, C, D, dt_bias, state, z=None):
        y, s, _ = O.scan_forward(x, dt, A, B, C, D, dt_bias, z, state, lengths)
        return (dy * y).sum() + (ds * s).sum()
    a = dict(args)
    g = O.scan_backward(a["x"], a["dt"], a["A"], a["B"], a["C"], dy, a["D"], a["dt_bias"], a.get("z"), a["state"], ds, lengths)
    _check_gradients(loss, args, g, list(args))


@pytest.mark.parametrize("lengths", [None, [4, 0, 1]])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [2, 4])
def test_conv_gradients(lengths, silu, K):
    rng = np.random.default_rng(4)
    B, T, C = 3, 4, 2
    r = lambda *s: rng.standard_normal(s)
    args = dict(x=r(B, T, C), w=r(C, K), bias=r(C), state=r(B, K - 1, C))
    dy, ds = r(B, T, C), r(B, K - 1, C)

    def loss(x, w, bias, state):
        y, s, _ = O.conv_forward(x, w, bias, state, lengths, silu)
        return (dy * y).sum() + (ds * s).sum()
    _check_gradients(loss, args, O.conv_backward(args["x"], args["w"], dy, args["bias"], args["state"], ds, lengths, silu), list(args))


@pytest.mark.parametrize("lengths", [None, [3, 0, 1]])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients(lengths, silu, gated):
    rng = np.random.default_rng(5)
    B, T, C, G = 3, 3, 6, 2
    r = lambda *s: rng.standard_normal(s)
    args = dict(x=r(B, T, C), weight=r(C), bias=r(C))
    if gated:
        args["gate"] = r(B, T, C)
    dy = r(B, T, C)

    def loss(x, weight, bias, gate=None):
        return (dy * O.norm_forward(x, G, weight, bias, gate, silu, 1e-2, lengths)[0]).sum()
    _check_gradients(loss, args, O.norm_backward(args["x"], G, dy, args["weight"], args["bias"], args.get("gate"), silu, 1e-2, lengths),
                     list(args))


def test_magnitudes_bound_the_values():
    rng = np.random.default_rng(6)
    r = lambda *s: rng.standard_normal(s)
    B, T, C, N = 2, 5, 4, 3
    a = (r(B, T, C), r(B, T, C), -np.exp(r(C, N)), r(B, T, 2, N), r(B, T, 2, N))
    kw = dict(D=r(C), z=r(B, T, C), state=r(B, C, N), lengths=[5, 3])
    for v, m in zip(O.scan_forward(*a, **kw), O.scan_forward(*a, **kw, mag=True)):
        assert np.all(np.abs(v) <= m + 1e-12)
    dy = r(B, T, C)
    g, m = O.scan_backward(*a, dy, **kw), O.scan_backward(*a, dy, **kw, mag=True)
    assert all(np.all(np.abs(g[k]) <= m[k] + 1e-12) for k in g)
    x, w = r(B, T, C), r(C, 3)
    g, m = O.conv_backward(x, w, dy), O.conv_backward(x, w, dy, mag=True)
    assert all(np.all(np.abs(g[k]) <= m[k] + 1e-12) for k in g)
    g, m = O.norm_backward(x, 2, dy, gate=r(B, T, C), silu=True), None
    m = O.norm_backward(x, 2, dy, mag=True)
    g = O.norm_backward(x, 2, dy)
    assert all(np.all(np.abs(g[k]) <= m[k] + 1e-12) for k in ("x", "weight", "bias"))
