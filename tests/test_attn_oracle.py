"""Pins of oracle/attn_oracle.py (CPU): hand-worked values, limits, and every gradient
against central differences of the forward."""
import numpy as np
import pytest

from oracle import attn_oracle as O
from tests.test_seq_oracle import _check_gradients, _close


def test_attention_by_hand():
    """One head, Dk = 2, Dv = 1, two tokens, decays 1/2 and 1/4."""
    q, k = np.array([[[[1.0, 0.0]], [[2.0, 1.0]]]]), np.array([[[[3.0, 1.0]], [[0.0, 5.0]]]])
    v, g = np.array([[[[2.0]], [[1.0]]]]), np.log(np.array([[[0.5], [0.25]]]))
    S0 = np.array([[[[4.0], [8.0]]]])
    # S_1 = (2 + 6, 4 + 2) = (8, 6); S_2 = (2 + 0, 1.5 + 5) = (2, 6.5)
    y, S, _ = O.attn_forward(q, k, v, g, scale=10.0, state=S0)
    _close(S, [[[[2.0], [6.5]]]], 1e-14)
    _close(y, [[[[80.0]], [[105.0]]]], 1e-14)


def test_attention_limits():
    rng = np.random.default_rng(0)
    B, T, H = 2, 7, 2
    q, k, v = (rng.standard_normal((B, T, H, n)) for n in (3, 3, 4))
    # no decay: the products of all earlier tokens
    y, _, _ = O.attn_forward(q, k, v, np.zeros(H))
    w = np.tril(np.ones((T, T)))[None, None] * np.einsum("bthd,bihd->bhti", q, k)
    _close(y, np.einsum("bhti,bihd->bthd", w, v), 1e-13)
    # the state is emptied at every token
    y, _, _ = O.attn_forward(q, k, v, np.full((B, T, H), -np.inf), state=rng.standard_normal((B, H, 3, 4)))
    _close(y, (q * k).sum(-1, keepdims=True) * v, 1e-13)
    # padding is as if it were not there
    q2, k2, v2 = q.copy(), k.copy(), v.copy()
    q2[1, 4:], k2[1, 4:], v2[1, 4:] = np.nan, np.inf, np.nan
    y, S, _ = O.attn_forward(q2, k2, v2, np.full(H, -0.3), lengths=[9, 4])
    y4, S4, _ = O.attn_forward(q[:, :4], k[:, :4], v[:, :4], np.full(H, -0.3))
    _close(y[1, :4], y4[1], 1e-14)
    _close(S[1], S4[1], 1e-14)
    assert np.all(y[1, 4:] == 0)
    # shared heads are repeated ones
    y, _, _ = O.attn_forward(q[:, :, :1], k, v[:, :, :1], np.full(H, -0.3))
    y2, _, _ = O.attn_forward(np.repeat(q[:, :, :1], 2, 2), k, np.repeat(v[:, :, :1], 2, 2), np.full(H, -0.3))
    _close(y, y2, 0)


def test_step_is_the_recurrence_on_a_pool():
    rng = np.random.default_rng(1)
    q, k, v, g, pool = (rng.standard_normal(s) for s in ((4, 1, 3), (4, 1, 3), (4, 2, 5), (4, 2), (6, 2, 3, 5)))
    y, after = O.attn_step(q, k, v, g, pool, [5, 2, 5, -1], scale=0.5)
    for b, s in ((0, 5), (1, 2)):
        y1, S1, _ = O.attn_forward(q[b][None, None], k[b][None, None], v[b][None, None], g[b][None, None], 0.5, pool[s][None])
        _close(y[b], y1[0, 0], 1e-14)
        _close(after[s], S1[0], 1e-14)
    assert np.all(y[2:] == 0)
    for s in (0, 1, 3, 4):
        assert np.all(after[s] == pool[s])


@pytest.mark.parametrize("lengths", [None, [4, 0, 2]])
@pytest.mark.parametrize("per_token", [True, False])
def test_attention_gradients(lengths, per_token):
    rng = np.random.default_rng(3)
    B, T, H = 3, 4, 4
    r = lambda *s: rng.standard_normal(s)
    args = dict(q=r(B, T, 2, 3), k=r(B, T, 1, 3), v=r(B, T, 4, 2), g=-np.exp(r(B, T, H) if per_token else r(H)), state=r(B, H, 3, 2))
    dy, ds = r(B, T, H, 2), r(B, H, 3, 2)

    def loss(q, k, v, g, state):
        y, s, _ = O.attn_forward(q, k, v, g, 0.7, state, lengths)
        return (dy * y).sum() + (ds * s).sum()
    grads = O.attn_backward(**{k: args[k] for k in "qkvg"}, dy=dy, scale=0.7, state=args["state"], dstate=ds, lengths=lengths)
    _check_gradients(loss, args, grads, ["q", "k", "v", "g", "state"])
    other = O.attn_backward(**{k: args[k] for k in "qkvg"}, dy=dy, scale=0.7, state=args["state"], dstate=ds, lengths=lengths, sums=True)
    _close(other["g"], grads["g"], 1e-12)


def test_magnitudes_bound_the_values():
    rng = np.random.default_rng(4)
    r = lambda *s: rng.standard_normal(s)
    q, k, v, g, dy, s, ds = r(2, 9, 2, 3), r(2, 9, 1, 3), r(2, 9, 2, 4), -np.exp(r(2, 9, 2)), r(2, 9, 2, 4), r(2, 2, 3, 4), r(2, 2, 3, 4)
    for sums in (False, True):
        a = O.attn_backward(q, k, v, g, dy, -0.5, s, ds, sums=sums)
        m = O.attn_backward(q, k, v, g, dy, -0.5, s, ds, mag=True, sums=sums)
        w = O.attn_backward(q, k, v, g, dy, -0.5, s, ds, mag=True, grow=(1e-3, 1e-3), sums=sums)
        for n in a:
            assert np.all(np.abs(a[n]) <= m[n] * (1 + 1e-12)) and np.all(m[n] <= w[n] * (1 + 1e-12)), n


def test_layer_norm():
    rng = np.random.default_rng(5)
    h = rng.standard_normal((2, 3, 7)) * 3 + 1
    y, mean, rstd = O.layer_forward(h, eps=1e-12)
    _close(y.mean(-1), np.zeros((2, 3)), 1e-12)
    _close(y.var(-1), np.ones((2, 3)), 1e-9)
    y, mean, rstd = O.layer_forward(h, eps=0.25, lengths=[3, 1])
    assert np.all(y[1, 1:] == 0) and np.all(mean[1, 1:] == 0) and np.all(rstd[1, 1:] == 2.0)


@pytest.mark.parametrize("lengths", [None, [2, 0]])
def test_layer_norm_gradients(lengths):
    rng = np.random.default_rng(6)
    r = lambda *s: rng.standard_normal(s)
    args = dict(h=r(2, 3, 5), weight=r(5), bias=r(5))
    dy, dh = r(2, 3, 5), r(2, 3, 5)
    there = np.ones((2, 3)) if lengths is None else np.arange(3)[None] < np.array(lengths)[:, None]

    def loss(h, weight, bias):
        return (dy * O.layer_forward(h, weight, bias, 1e-2, lengths)[0]).sum() + (dh * h * there[..., None]).sum()
    grads = O.layer_backward(args["h"], dy, args["weight"], dh, 1e-2, lengths)
    _check_gradients(loss, args, grads, ["h", "weight", "bias"])
