"""GPU parity of the short causal convolution against the fp64 oracle."""
import numpy as np
import pytest

from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def M():
    from linear_rnn_sequence_wkv7_amd import shortconv
    return shortconv


def make(seed, B, T, C, K, dtype, bias=True, state=True):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)
    return dict(x=S.as_dtype(r(B, T, C), dtype), w=r(C, K).astype(np.float32), bias=r(C).astype(np.float32) if bias else None,
                state=S.as_dtype(r(B, K - 1, C), dtype) if state else None, dy=S.as_dtype(r(B, T, C), dtype),
                dstate=r(B, K - 1, C).astype(np.float32) if state else None)


def lens(lengths):
    return None if lengths is None else torch().tensor(lengths, dtype=torch().int32, device="cuda")


CASES = [
    # B, T, C, K, dtype, lengths, bias, state
    (1, 1, 1, 2, "f32", None, False, False),
    (2, 2, 3, 4, "bf16", None, True, True),
    (3, 3, 8, 4, "f32", [3, 0, 1], True, True),
    (4, 7, 16, 3, "bf16", [7, 2, 1, 0], True, True),
    (1, 8, 24, 2, "f32", None, True, True),
    (2, 33, 10, 4, "f32", [33, 9], True, True),
    (2, 100, 72, 4, "bf16", None, False, True),
    (1, 129, 7, 3, "bf16", None, True, False),
    (5, 37, 514, 4, "f32", [37, 36, 8, 2, 0], True, True),
    (16, 256, 4096, 4, "bf16", None, True, True),      # long runs
    (2, 0, 8, 4, "f32", None, True, True),
    (2, 5, 0, 4, "f32", None, True, True),
    (0, 5, 8, 4, "f32", None, True, True),
]
IDS = ["B{}_T{}_C{}_K{}_{}".format(*c[:5]) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("act", ["silu", "none"])
def test_forward(case, act):
    B, T, C, K, dtype, lengths, bias, state = case
    m = make(T + C, B, T, C, K, dtype, bias, state)
    (y_ref, s_ref), (y_tol, _) = S.conv_bounds(m["x"], m["w"], m["bias"], m["state"], lengths, act == "silu")
    y, s = M().shortconv_forward(to_dev(m["x"]), to_dev(m["w"]), bias=to_dev(m["bias"]), state=to_dev(m["state"]),
                                 lengths=lens(lengths), act=act, y_dtype="f32" if T % 2 else None)
    torch().cuda.synchronize()
    S.check("y", to_host(y), y_ref, y_tol, bf16=y.dtype == torch().bfloat16)
    np.testing.assert_array_equal(to_host(s), s_ref)


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("act", ["silu", "none"])
def test_backward(case, act):
    B, T, C, K, dtype, lengths, bias, state = case
    if B * T * C > 1 << 20:
        B, T = 2, 300
    m = make(T + C + 1, B, T, C, K, dtype, bias, state)
    ref, tol = S.conv_bounds(m["x"], m["w"], m["bias"], m["state"], lengths, act == "silu", m["dy"], m["dstate"])
    g = M().shortconv_backward(to_dev(m["x"]), to_dev(m["w"]), to_dev(m["dy"]), bias=to_dev(m["bias"]), state=to_dev(m["state"]),
                               dstate=to_dev(m["dstate"]), lengths=lens(lengths), act=act)
    torch().cuda.synchronize()
    for k in ref:
        if g[k] is None:
            assert k == "bias" and not bias
            continue
        S.check("d" + k, to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == torch().bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_every_small_size(K, dtype):
    """Channels and tokens around the widths of a load, a run of tokens and the taps."""
    for C in (1, 2, 3, 4, 6, 7, 8, 12, 15, 16, 24, 40, 260):
        for T in (1, 2, 3, 4, 5, 7, 8, 9, 17, 33):
            lengths = [T, max(0, T - K + 1)]
            m = make(C * T, 2, T, C, K, dtype, C % 3 != 0, T % 2 == 0)
            (y_ref, s_ref), (y_tol, _) = S.conv_bounds(m["x"], m["w"], m["bias"], m["state"], lengths, True)
            kw = dict(bias=to_dev(m["bias"]), state=to_dev(m["state"]), lengths=lens(lengths), act="silu")
            y, s = M().shortconv_forward(to_dev(m["x"]), to_dev(m["w"]), **kw)
            S.check(f"y {C} {T}", to_host(y), y_ref, y_tol, bf16=dtype == "bf16")
            np.testing.assert_array_equal(to_host(s), s_ref)
            ref, tol = S.conv_bounds(m["x"], m["w"], m["bias"], m["state"], lengths, True, m["dy"], m["dstate"])
            g = M().shortconv_backward(to_dev(m["x"]), to_dev(m["w"]), to_dev(m["dy"]), dstate=to_dev(m["dstate"]), **kw)
            for k in ref:
                if g[k] is not None:
                    S.check(f"d{k} {C} {T}", to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == torch().bfloat16)


def test_padding_values_do_not_matter():
    B, T, C, K = 3, 21, 16, 4
    lengths = [10, 0, 2]
    m = make(1, B, T, C, K, "f32")
    out = []
    for fill in (np.nan, 0.0):
        x, dy = m["x"].copy(), m["dy"].copy()
        for b, n in enumerate(lengths):
            x[b, n:], dy[b, n:] = fill, fill
        kw = dict(bias=to_dev(m["bias"]), state=to_dev(m["state"]), lengths=lens(lengths))
        y, s = M().shortconv_forward(to_dev(x), to_dev(m["w"]), **kw)
        g = M().shortconv_backward(to_dev(x), to_dev(m["w"]), to_dev(dy), dstate=to_dev(m["dstate"]), **kw)
        torch().cuda.synchronize()
        out.append({"y": to_host(y), "s": to_host(s), **{k: to_host(v) for k, v in g.items()}})
    for k in out[0]:
        np.testing.assert_array_equal(out[0][k], out[1][k], err_msg=k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,K", [(64, 4), (35, 4), (10, 3), (2050, 2)])
def test_step(C, K, dtype):
    B, Sp = 7, 9
    m = make(C, B, 1, C, K, dtype)
    pool = S.as_dtype(np.random.default_rng(C).standard_normal((Sp, K - 1, C)), dtype)
    index = [4, -1, 0, 8, 4, 9, 2]
    st = to_dev(pool)
    y = M().shortconv_step(to_dev(m["x"][:, 0]), to_dev(m["w"]), st, bias=to_dev(m["bias"]),
                           state_index=torch().tensor(index, dtype=torch().int32, device="cuda"))
    torch().cuda.synchronize()
    rows = [0, 2, 3, 6]
    at = [index[r] for r in rows]
    (y_ref, s_ref), (y_tol, _) = S.conv_bounds(m["x"][rows], m["w"], m["bias"], pool[at], None, True)
    S.check("y", to_host(y)[rows], y_ref[:, 0], y_tol[:, 0], bf16=dtype == "bf16")
    new, old = to_host(st), to_host(to_dev(pool))
    np.testing.assert_array_equal(new[at], s_ref)
    assert np.all(to_host(y)[[1, 4, 5]] == 0)
    np.testing.assert_array_equal(new[[1, 3, 5, 6, 7]], old[[1, 3, 5, 6, 7]])


@pytest.mark.parametrize("lengths", [None, [2, 0, 1, 5]])
def test_in_place_state_and_steps(lengths):
    """The state moved in place, and steps after it as in one long call."""
    B, T, C, K = 4, 5, 32, 4
    m = make(3, B, T, C, K, "bf16")
    x, w, bias = to_dev(m["x"]), to_dev(m["w"]), to_dev(m["bias"])
    _, s1 = M().shortconv_forward(x, w, bias=bias, state=to_dev(m["state"]), lengths=lens(lengths))
    st = to_dev(m["state"])
    y2, s2 = M().shortconv_forward(x, w, bias=bias, state=st, state_out=st, lengths=lens(lengths))
    assert s2 is st and torch().equal(s1, s2)
    if lengths is None:
        st = to_dev(m["state"])
        ys = [M().shortconv_step(x[:, t].contiguous(), w, st, bias=bias) for t in range(T)]
        torch().cuda.synchronize()
        assert torch().equal(st, s1)
        assert torch().equal(torch().stack(ys, 1), y2)
