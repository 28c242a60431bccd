"""GPU parity of the group norm against the fp64 oracle."""
import numpy as np
import pytest

from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def M():
    from linear_rnn_sequence_wkv7_amd import groupnorm
    return groupnorm


def make(seed, B, T, C, dtype, affine=True, gate=True, mean=0.3):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)
    return dict(x=S.as_dtype(r(B, T, C) * 0.8 + mean, dtype), dy=S.as_dtype(r(B, T, C), dtype),
                weight=(1 + 0.3 * r(C)).astype(np.float32) if affine else None,
                bias=(0.3 * r(C)).astype(np.float32) if affine else None,
                gate=S.as_dtype(r(B, T, C), dtype) if gate else None)


def lens(lengths):
    return None if lengths is None else torch().tensor(lengths, dtype=torch().int32, device="cuda")


CASES = [
    # B, T, C, G, dtype, lengths, affine, gate, act
    (5, 1, 64, 1, "f32", None, True, True, "none"),
    (9, 1, 256, 4, "bf16", None, True, True, "none"),
    (3, 1, 128, 16, "f32", None, False, False, "silu"),
    (4, 1, 1024, 2, "bf16", None, True, False, "silu"),
    (2, 1, 1040, 65, "bf16", [1, 0], True, True, "silu"),
    (3, 1, 2432, 38, "bf16", None, True, True, "none"),
    (700, 1, 320, 5, "bf16", None, True, True, "none"),
    (4100, 1, 64, 2, "f32", None, True, False, "none"),
    (6, 1, 30, 3, "f32", [1, 1, 0, 1, 1, 1], True, True, "silu"),
    (5, 1, 1626, 6, "bf16", None, True, True, "none"),
    (5, 1, 1999, 1, "f32", None, True, True, "silu"),
    (3, 1, 24, 1, "f32", None, True, True, "none"),
    (2, 1, 5, 5, "f32", None, True, False, "none"),
    (2, 1, 9000, 2, "bf16", None, True, True, "none"),
    (2, 2, 16, 2, "f32", None, True, True, "silu"),
    (3, 63, 24, 3, "bf16", [63, 1, 0], True, True, "silu"),
    (2, 130, 60, 4, "f32", [130, 65], True, False, "silu"),
    (1, 300, 33, 11, "f32", None, True, True, "none"),
    (2, 64, 1024, 8, "bf16", None, False, False, "none"),
    (2, 65, 10, 2, "bf16", None, True, True, "silu"),
    (2, 1531, 96, 3, "f32", [1531, 700], True, True, "silu"),      # a group of a sequence in a workgroup's registers
    (2, 1100, 28, 2, "bf16", None, True, True, "none"),
    (2, 3000, 96, 2, "f32", [2999, 3000], True, True, "silu"),     # and past them
    (1, 700, 1044, 1, "bf16", None, True, False, "silu"),
    (1, 1000, 514, 1, "f32", None, True, True, "none"),
    (1, 130, 1999, 1, "bf16", [77], False, True, "silu"),
]
IDS = ["B{}_T{}_C{}_G{}_{}_{}".format(*c[:5], c[8]) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(case):
    B, T, C, G, dtype, lengths, affine, gate, act = case
    m = make(T + C, B, T, C, dtype, affine, gate)
    (y_ref, m_ref, r_ref), (y_tol, m_tol, r_tol) = S.norm_bounds(m["x"], G, m["weight"], m["bias"], m["gate"], act == "silu", EPS, lengths)
    kw = dict(weight=to_dev(m["weight"]), bias=to_dev(m["bias"]), gate=to_dev(m["gate"]), act=act, eps=EPS, lengths=lens(lengths))
    y, mean, rstd = M().groupnorm_forward(to_dev(m["x"]), G, **kw, y_dtype="f32" if C % 4 else None)
    y2, none, _ = M().groupnorm_forward(to_dev(m["x"]), G, **kw, y_dtype="f32" if C % 4 else None, return_stats=False)
    torch().cuda.synchronize()
    S.check("y", to_host(y), y_ref, y_tol, bf16=y.dtype == torch().bfloat16)
    S.check("mean", to_host(mean), m_ref, m_tol)
    S.check("rstd", to_host(rstd), r_ref, r_tol)
    assert none is None and torch().equal(y, y2)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    B, T, C, G, dtype, lengths, affine, gate, act = case
    m = make(T + C + 1, B, T, C, dtype, affine, gate)
    ref, tol = S.norm_bounds(m["x"], G, m["weight"], m["bias"], m["gate"], act == "silu", EPS, lengths, dy=m["dy"])
    kw = dict(weight=to_dev(m["weight"]), bias=to_dev(m["bias"]), gate=to_dev(m["gate"]), act=act, lengths=lens(lengths))
    x = to_dev(m["x"])
    _, mean, rstd = M().groupnorm_forward(x, G, eps=EPS, **kw)
    g = M().groupnorm_backward(x, G, to_dev(m["dy"]), mean, rstd, **kw)
    torch().cuda.synchronize()
    for k in ref:
        if g[k] is None:
            assert (k in ("weight", "bias") and not affine) or (k == "gate" and not gate)
            continue
        S.check("d" + k, to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == torch().bfloat16)


@pytest.mark.parametrize("B,T,C,G", [(6, 1, 128, 2), (6, 1, 21, 3), (3, 40, 32, 2), (2, 70, 15, 3)])
def test_variance_far_from_zero(B, T, C, G):
    """Values of spread 1 around 1000: the differences from the mean carry the variance, so it keeps
    the accuracy that the inputs have."""
    m = make(B + C, B, T, C, "f32", mean=1000.0)
    (y_ref, m_ref, r_ref), (y_tol, m_tol, r_tol) = S.norm_bounds(m["x"], G, m["weight"], m["bias"], None, False, EPS, None)
    y, mean, rstd = M().groupnorm_forward(to_dev(m["x"]), G, weight=to_dev(m["weight"]), bias=to_dev(m["bias"]), eps=EPS)
    S.check("y", to_host(y), y_ref, y_tol)
    S.check("mean", to_host(mean), m_ref, m_tol)
    # the variance of differences that are off by e is off by e^2 at the most: 60 U 1000 squared is far below 1e-4
    S.check("rstd", to_host(rstd), r_ref, 1e-4 * r_ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 5, 33])
def test_every_small_group(T, dtype):
    """Groups of 1 to 72 channels and some around the widths of a wave, with and without a gate."""
    for Cg in [*range(1, 73), 126, 128, 130, 255, 257, 514]:
        G, B = 1 + Cg % 3, 3
        act, lengths = ("silu", [T, 0, (T + 1) // 2]) if Cg % 2 else ("none", None)
        m = make(Cg, B, T, G * Cg, dtype, True, Cg % 4 < 2)
        (y_ref, m_ref, r_ref), (y_tol, m_tol, r_tol) = S.norm_bounds(m["x"], G, m["weight"], m["bias"], m["gate"], act == "silu", EPS, lengths)
        kw = dict(weight=to_dev(m["weight"]), bias=to_dev(m["bias"]), gate=to_dev(m["gate"]), act=act, lengths=lens(lengths))
        x = to_dev(m["x"])
        y, mean, rstd = M().groupnorm_forward(x, G, eps=EPS, **kw)
        S.check(f"y {Cg}", to_host(y), y_ref, y_tol, bf16=dtype == "bf16")
        S.check(f"mean {Cg}", to_host(mean), m_ref, m_tol)
        S.check(f"rstd {Cg}", to_host(rstd), r_ref, r_tol)
        ref, tol = S.norm_bounds(m["x"], G, m["weight"], m["bias"], m["gate"], act == "silu", EPS, lengths, dy=m["dy"])
        g = M().groupnorm_backward(x, G, to_dev(m["dy"]), mean, rstd, **kw)
        for k in ref:
            if g[k] is not None:
                S.check(f"d{k} {Cg}", to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == torch().bfloat16)


def test_constant_groups():
    """A group of equal values has variance 0: y is act(bias) gate, rstd 1 / sqrt(eps)."""
    x = np.full((3, 1, 64), 2.0, np.float32)
    b = np.arange(64, dtype=np.float32)
    y, mean, rstd = M().groupnorm_forward(to_dev(x), 4, bias=to_dev(b), eps=0.25)
    np.testing.assert_array_equal(to_host(y)[:, 0], np.broadcast_to(b, (3, 64)))
    np.testing.assert_array_equal(to_host(mean), np.full((3, 4), 2.0))
    np.testing.assert_array_equal(to_host(rstd), np.full((3, 4), 2.0))


@pytest.mark.parametrize("T,C,G", [(1, 64, 2), (1, 30, 2), (9, 24, 3)])
def test_padding_values_do_not_matter(T, C, G):
    B = 3
    lengths = [T, 0, T // 2]
    m = make(2, B, T, C, "f32")
    out = []
    for fill in (np.nan, 0.0):
        x, dy, gate = m["x"].copy(), m["dy"].copy(), m["gate"].copy()
        for b, n in enumerate(lengths):
            x[b, n:], dy[b, n:], gate[b, n:] = fill, fill, fill
        kw = dict(weight=to_dev(m["weight"]), bias=to_dev(m["bias"]), gate=to_dev(gate), act="silu", lengths=lens(lengths))
        y, mean, rstd = M().groupnorm_forward(to_dev(x), G, **kw)
        g = M().groupnorm_backward(to_dev(x), G, to_dev(dy), mean, rstd, **kw)
        torch().cuda.synchronize()
        out.append({"y": to_host(y), "mean": to_host(mean), "rstd": to_host(rstd), **{k: to_host(v) for k, v in g.items()}})
    for k in out[0]:
        np.testing.assert_array_equal(out[0][k], out[1][k], err_msg=k)


def test_empty():
    t = torch()
    y, mean, rstd = M().groupnorm_forward(t.empty(2, 0, 16, device="cuda"), 4, eps=0.25)
    assert y.numel() == 0 and bool((mean == 0).all()) and bool((rstd == 2).all())
    w = t.ones(16, device="cuda")
    g = M().groupnorm_backward(t.empty(0, 3, 16, device="cuda"), 4, t.empty(0, 3, 16, device="cuda"), t.empty(0, 4, device="cuda"),
                               t.empty(0, 4, device="cuda"), weight=w, bias=w)
    assert bool((g["weight"] == 0).all()) and bool((g["bias"] == 0).all())


def test_more_groups_than_a_launch_of_whole_workgroups_takes():
    """2^22 groups of two values.  With u = 2^-24 and M the larger value: the mean is off by 2 u M, a difference by 3 u M,
    their square's mean by 6 u M |d| + 4 u d^2; so y = d rstd by 6 u M rstd + 4 u; 16 u (M rstd + 1) covers it."""
    t = torch()
    x = t.randn(1 << 21, 2, 2, device="cuda")
    y, mean, rstd = M().groupnorm_forward(x, 2, eps=EPS)
    xd = x.double()
    d = xd - xd.mean(1, keepdim=True)
    r = 1 / t.sqrt((d * d).mean(1, keepdim=True) + EPS)
    tol = 16 * 2.0 ** -24 * (xd.abs().amax(1, keepdim=True) * r + 1)
    assert bool(((y.double() - d * r).abs() <= tol).all())
