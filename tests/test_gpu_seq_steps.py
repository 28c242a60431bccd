"""Single tokens of many rows at once: the forms of the step kernels in which a
workgroup has several rows, with repeated, missing and out-of-range states among the
rows of one workgroup and of different ones, and rows that are no multiple of them."""
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


def indices(rng, B, Sp):
    """Rows' states: at random, runs of one state inside four rows and across them, none (below 0, from Sp on)."""
    index = rng.integers(-2, Sp + 2, B).astype(np.int32)
    for at, pattern in ((0, (3, 3, 3, 3)), (4, (5, -1, 5, 6)), (8, (3, 7, 7, 9)), (12, (-1, -1, -1, -1)), (16, (Sp, 10, -7, 10)),
                        (21, (11, 11)), (B - 3, (12, 0, 12)), (B - 1, (Sp - 1,))):
        index[at:at + len(pattern)] = pattern
    first, seen = [], set()
    for b, s in enumerate(index.tolist()):
        if 0 <= s < Sp and s not in seen:
            seen.add(s)
            first.append(b)
    return index, np.array(first)


def check_rows(y, st, old, index, first, y_ref, y_tol, bf16):
    S.check("y", y[first], y_ref, y_tol, bf16=bf16)
    assert np.all(np.delete(y, first, 0) == 0)
    left = np.setdiff1d(np.arange(len(old)), index[first])
    assert len(left)
    np.testing.assert_array_equal(st[left], old[left])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,N,G", [(1027, 256, 16, 1), (1025, 250, 16, 5), (1030, 900, 4, 3), (2051, 255, 7, 1), (1027, 100, 20, 1), (1026, 64, 64, 2)])
def test_scan(B, C, N, G, dtype):
    lanes = 1 if N <= 4 else 2 if N <= 8 else 4 if N <= 16 else 8 if N <= 32 else 16
    assert -(-C * lanes // 256) * B >= 4096 and B % 4   # four rows to a workgroup, and some left
    rng = np.random.default_rng(B + N)
    Sp = B // 2
    x = S.scan_inputs(C + N, B, 1, C, N, G, dtype, step=True)
    pool = rng.standard_normal((Sp, C, N)).astype(np.float32)
    index, first = indices(rng, B, Sp)
    from linear_rnn_sequence_wkv7_amd import ssm
    d = {k: to_dev(v) for k, v in x.items()}
    st = to_dev(pool)
    args, kw = (d["x"], d["dt"], d["A"], d["Bm"], d["Cm"]), dict(D=d["D"], dt_bias=d["dt_bias"], z=d["z"])
    y = ssm.ssm_step(*args, st, state_index=to_dev(index), **kw)
    torch().cuda.synchronize()
    pick = {k: (v[first][:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in x.items()}
    pick["state"] = pool[index[first]]
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(pick, 1, None, True)
    new = to_host(st)
    check_rows(to_host(y), new, pool, index, first, y_ref[:, 0], y_tol[:, 0], dtype == "bf16")
    S.check("state", new[index[first]], s_ref, s_tol)
    # without an index: row b on state b, the states behind the last row left as they were
    more = rng.standard_normal((B + 3, C, N)).astype(np.float32)
    st = to_dev(more)
    y = ssm.ssm_step(*args, st, **kw)
    torch().cuda.synchronize()
    last = {k: (v[-5:][:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in x.items()}
    last["state"] = more[B - 5:B]
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(last, 1, None, True)
    S.check("y of the last rows", to_host(y)[-5:], y_ref[:, 0], y_tol[:, 0], bf16=dtype == "bf16")
    S.check("their states", to_host(st)[B - 5:B], s_ref, s_tol)
    np.testing.assert_array_equal(to_host(st)[B:], more[B:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,K", [(515, 24, 4), (513, 7, 3), (601, 10, 2), (517, 12, 4), (301, 2056, 4)])
def test_convolution(B, C, K, dtype):
    slots = C // (8 if C % 8 == 0 else 4 if C % 4 == 0 else 2 if C % 2 == 0 else 1)
    assert -(-slots // 256) * B >= 512 and B % 2   # two rows to a workgroup, and one left
    rng = np.random.default_rng(B + C)
    r = lambda *s: rng.standard_normal(s)
    Sp = B // 2
    x, pool = S.as_dtype(r(B, C), dtype), S.as_dtype(r(Sp, K - 1, C), dtype)
    w, bias = r(C, K).astype(np.float32), r(C).astype(np.float32)
    index, first = indices(rng, B, Sp)
    from linear_rnn_sequence_wkv7_amd import shortconv
    st = to_dev(pool)
    old = to_host(st)
    y = shortconv.shortconv_step(to_dev(x), to_dev(w), st, bias=to_dev(bias), state_index=to_dev(index))
    torch().cuda.synchronize()
    (y_ref, s_ref), (y_tol, _) = S.conv_bounds(x[first][:, None], w, bias, pool[index[first]], None, True)
    new = to_host(st)
    check_rows(to_host(y), new, old, index, first, y_ref[:, 0], y_tol[:, 0], dtype == "bf16")
    np.testing.assert_array_equal(new[index[first]], s_ref)
    # without an index
    more = S.as_dtype(r(B + 3, K - 1, C), dtype)
    st = to_dev(more)
    old = to_host(st)
    y = shortconv.shortconv_step(to_dev(x), to_dev(w), st, bias=to_dev(bias))
    torch().cuda.synchronize()
    (y_ref, s_ref), (y_tol, _) = S.conv_bounds(x[:, None], w, bias, more[:B], None, True)
    S.check("y", to_host(y), y_ref[:, 0], y_tol[:, 0], bf16=dtype == "bf16")
    np.testing.assert_array_equal(to_host(st)[:B], s_ref)
    np.testing.assert_array_equal(to_host(st)[B:], old[B:])
