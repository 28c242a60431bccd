"""The layer norm over a residual stream on the GPU against the fp64 oracle: rows of every width and phase, types,
padding, outputs in place."""
import numpy as np
import pytest

from tests import attn_util as A
from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def mod():
    from linear_rnn_sequence_wkv7_amd import layernorm
    return layernorm


def is_bf16(t):
    return t.dtype == torch().bfloat16


def run(x, y_dtype, dh=True, lengths=None, eps=1e-5, weight=True, bias=True, x_dtype=None, seed=3):
    """Forward and backward, both compared."""
    rng = np.random.default_rng(seed)
    d = {k: to_dev(v) for k, v in x.items()}
    w, b = (x["weight"] if weight else None), (x["bias"] if bias else None)
    kw = dict(weight=d["weight"] if weight else None, bias=d["bias"] if bias else None, lengths=to_dev(lengths))
    y, h, mean, rstd = mod().layernorm_forward(d["x"], residual=d["residual"], eps=eps, y_dtype=y_dtype, **kw)
    href = A.stream(x)
    B, T, C = href.shape
    there = np.ones((B, T), bool) if lengths is None else np.arange(T)[None] < np.asarray(lengths)[:, None]
    hd = to_dev(np.where(there[..., None], href, np.zeros((), href.dtype)))
    if d["residual"] is None:
        assert h is d["x"]
    else:
        assert torch().equal(h, hd)
    (y_ref, m_ref, r_ref), (y_tol, m_tol, r_tol), _ = A.norm_bounds(href, w, b, eps, lengths)
    S.check("y", to_host(y), y_ref, y_tol, bf16=is_bf16(y))
    S.check("mean", to_host(mean), m_ref, m_tol)
    S.check("rstd", to_host(rstd), r_ref, r_tol)
    dy = S.as_dtype(rng.standard_normal((B, T, C)), y_dtype)
    gh = S.as_dtype(rng.standard_normal((B, T, C)), "bf16" if is_bf16(h) else "f32") if dh else None
    g = mod().layernorm_backward(h, to_dev(dy), mean, rstd, dh=to_dev(gh), x_dtype=x_dtype, **kw)
    torch().cuda.synchronize()
    ref, tol = A.norm_grad_bounds(href, dy, w, gh, eps, lengths)
    S.check("dh", to_host(g["h"]), ref["h"], tol["h"], bf16=is_bf16(h))
    S.check("dx", to_host(g["x"]), ref["h"], tol["h"], bf16=is_bf16(g["x"]))
    for n, there in (("weight", weight), ("bias", bias)):
        if there:
            S.check("d" + n, to_host(g[n]), ref[n], tol[n])
        else:
            assert g[n] is None
    return y, h, mean, rstd, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 2, 5, 7, 8, 9, 63, 64, 65, 100, 504, 505, 512, 513, 1001, 1024, 1030, 2041, 2042, 2048, 2050, 4096, 4100, 8185, 8186, 8192,
                               8200, 16384, 16392, 17001])
def test_widths(C, dtype):
    run(A.norm_inputs(C, 2, 9, C, dtype, dtype), dtype)


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 8, 9, 31, 33, 600, 5000])
@pytest.mark.parametrize("C", [24, 61])
def test_rows(rows, C):
    """Fewer and more rows than are taken at once, also where rows differ in phase."""
    run(A.norm_inputs(rows, 1, rows, C, "bf16", "bf16"), "bf16")


@pytest.mark.parametrize("C", [96, 97, 3000, 9000])
@pytest.mark.parametrize("x_dtype,h_dtype,y_dtype", [("bf16", "f32", "bf16"), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", "bf16"), ("bf16", "bf16", "f32")])
def test_types(x_dtype, h_dtype, y_dtype, C):
    y, h, _, _, g = run(A.norm_inputs(C, 2, 11, C, x_dtype, h_dtype), y_dtype, x_dtype=x_dtype)
    names = {"f32": torch().float32, "bf16": torch().bfloat16}
    assert (y.dtype, h.dtype, g["h"].dtype, g["x"].dtype) == tuple(names[n] for n in (y_dtype, h_dtype, h_dtype, x_dtype))


@pytest.mark.parametrize("weight,bias,dh,residual", [(False, False, False, False), (True, False, True, True), (False, True, False, True), (True, True, False, False)])
@pytest.mark.parametrize("C", [160, 161, 20000])
def test_optional_inputs(C, weight, bias, dh, residual):
    run(A.norm_inputs(C, 2, 5, C, "f32", "f32", residual), "f32", dh=dh, weight=weight, bias=bias)


@pytest.mark.parametrize("C", [40, 41, 2048, 16390])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding(C, dtype):
    """Whatever padding holds, in the forward and, with its statistics, in the backward."""
    t = torch()
    lengths = np.array([6, 0, 2, 9, -3], np.int32)
    x = A.norm_inputs(C, 5, 6, C, dtype, dtype)
    y, h, mean, rstd, g = run(x, dtype, lengths=np.clip(lengths, 0, 6))
    nan = 0x7FC0 if dtype == "bf16" else np.nan
    bad = {k: v.copy() for k, v in x.items()}
    for b, n in enumerate(np.clip(lengths, 0, 6)):
        bad["x"][b, n:] = nan
        bad["residual"][b, n:] = nan
    d = {k: to_dev(v) for k, v in bad.items()}
    kw = dict(weight=d["weight"], bias=d["bias"], lengths=to_dev(lengths))
    y2, h2, m2, r2 = mod().layernorm_forward(d["x"], residual=d["residual"], **kw)
    assert t.equal(y, y2) and t.equal(h, h2) and t.equal(mean, m2) and t.equal(rstd, r2)
    rng = np.random.default_rng(3)
    dy, gh = to_dev(S.as_dtype(rng.standard_normal(x["x"].shape), dtype)), to_dev(S.as_dtype(rng.standard_normal(x["x"].shape), dtype))
    for b, n in enumerate(np.clip(lengths, 0, 6)):
        for a in (h2, dy, gh, m2, r2):
            a[b, n:] = float("nan")
    g2 = mod().layernorm_backward(h2, dy, m2, r2, dh=gh, **kw)
    for n in g:
        assert t.equal(g[n], g2[n]), n


def test_nothing_to_compute():
    t = torch()
    z = lambda *s: t.zeros(s, device="cuda")
    y, h, mean, rstd = mod().layernorm_forward(z(2, 3, 0), eps=0.25)
    assert mean.shape == (2, 3) and t.all(mean == 0) and t.all(rstd == 2.0)
    y, h, mean, rstd = mod().layernorm_forward(z(0, 3, 8), weight=z(8))
    g = mod().layernorm_backward(h, y, mean, rstd, weight=z(8), bias=z(8), grads={"weight": t.full((8,), 7.0, device="cuda")})
    assert t.all(g["weight"] == 0) and t.all(g["bias"] == 0)


@pytest.mark.parametrize("C", [130, 131, 4096, 20001])
def test_the_stream_in_place(C):
    """h in residual's place and the gradient in dh's."""
    t = torch()
    x = A.norm_inputs(C, 2, 30, C, "bf16", "bf16")
    y, h, mean, rstd, g = run(x, "bf16")
    d = {k: to_dev(v) for k, v in x.items()}
    kw = dict(weight=d["weight"], bias=d["bias"])
    y2, h2, _, _ = mod().layernorm_forward(d["x"], residual=d["residual"], h=d["residual"], return_stats=False, **kw)
    assert h2 is d["residual"] and t.equal(h2, h) and t.equal(y2, y)
    rng = np.random.default_rng(3)
    dy, gh = (to_dev(S.as_dtype(rng.standard_normal(x["x"].shape), "bf16")) for _ in range(2))
    g2 = mod().layernorm_backward(h, dy, mean, rstd, dh=gh, grads={"h": gh}, **kw)
    assert g2["h"] is gh and t.equal(gh, g["h"]) and t.equal(g2["weight"], g["weight"])


def test_large_means_and_equal_rows():
    """Rows far from zero (the variance is of the differences from the mean), rows of one value, huge rows."""
    rng = np.random.default_rng(0)
    x = A.norm_inputs(1, 1, 40, 1000, "f32", "f32", residual=False)
    x["x"][0, :10] += 1000.0
    x["x"][0, 10:20] = 3.0
    x["x"][0, 20:30] *= 1e15
    run(x, "f32")
