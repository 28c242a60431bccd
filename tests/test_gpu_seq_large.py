"""The scan, the convolution and the group norm on arrays of more than 2^31 elements
(more than 2^32 bytes), where every offset of the last rows needs 64 bits: the last
sequence, or the last tokens of a long one, against the oracle.  Where gradients are
summed over the batch, only the last sequence's dy is not 0 (adding 0 rounds nothing)."""
import numpy as np
import pytest

from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch

pytestmark = pytest.mark.gpu

B, T, C = 8200, 64, 4096
assert B * T * C > 1 << 31


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield
    torch().cuda.empty_cache()


def normal(seed, *shape, dtype="bf16"):
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(seed)
    return t.randn(shape, generator=gen, device="cuda", dtype=t.bfloat16 if dtype == "bf16" else t.float32)


def host(t):
    """bf16 bit patterns or fp32 values of a small tensor, as the oracle takes them."""
    tt = torch()
    t = t.contiguous()
    return t.view(tt.int16).cpu().numpy().view(np.uint16) if t.dtype == tt.bfloat16 else t.cpu().numpy()


def check(what, got, ref, tol):
    S.check(what, to_host(got.contiguous()), ref, tol, bf16=got.dtype == torch().bfloat16)


def parameters(N):
    rng = np.random.default_rng(N)
    A = -np.exp(rng.uniform(-3, 1.2, (C, N))).astype(np.float32)
    return A, rng.standard_normal(C).astype(np.float32), (rng.standard_normal(C) * 0.5 - 1).astype(np.float32)


def scan_part(x, b, grp, G):
    """Sequence b, channels of one group, as an oracle problem."""
    cs = slice(grp * (C // G), (grp + 1) * (C // G))
    p = {k: host(x[k][b:b + 1, :, cs]) for k in ("x", "dt", "z")}
    p.update({k: host(x[k][b:b + 1, :, grp:grp + 1]) for k in ("Bm", "Cm")})
    p.update(A=x["A"][cs], D=x["D"][cs], dt_bias=x["dt_bias"][cs], state=host(x["state"][b:b + 1, cs]))
    return p, cs


def scan_tensors(N, G):
    x = {k: normal(i, B, T, C) for i, k in enumerate(("x", "dt", "z"))}
    x.update({k: normal(i + 7, B, T, G, N) for i, k in enumerate(("Bm", "Cm"))})
    x["A"], x["D"], x["dt_bias"] = parameters(N)
    x["state"] = normal(11, B, C, N, dtype="f32")
    return x, (x["x"], x["dt"], to_dev(x["A"]), x["Bm"], x["Cm"]), dict(D=to_dev(x["D"]), dt_bias=to_dev(x["dt_bias"]), z=x["z"], state=x["state"])


def test_scan_forward():
    from linear_rnn_sequence_wkv7_amd import ssm
    N, G = 16, 256   # B and C past 2^31 elements too
    x, a, kw = scan_tensors(N, G)
    assert x["Bm"].numel() > 1 << 31
    y, s = ssm.ssm_forward(*a, **kw)
    torch().cuda.synchronize()
    for b, grp in ((0, 0), (B - 1, G - 1), (B - 2, 17)):
        p, cs = scan_part(x, b, grp, G)
        (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(p, T, None, True, Cg=C // G)
        check("y", y[b:b + 1, :, cs], y_ref, y_tol)
        check("state", s[b:b + 1, cs], s_ref, s_tol)


def test_scan_backward():
    from linear_rnn_sequence_wkv7_amd import ssm
    N, G = 16, 64
    x, a, kw = scan_tensors(N, G)
    dy = torch().zeros(B, T, C, device="cuda", dtype=torch().bfloat16)
    dy[B - 1] = normal(3, T, C)
    g = ssm.ssm_backward(*a, dy, **kw)
    torch().cuda.synchronize()
    for grp in (G - 1, 5):
        p, cs = scan_part(x, B - 1, grp, G)
        ref, tol = S.scan_bounds(p, T, None, True, dy=host(dy[B - 1:, :, cs]), Cg=C // G)
        for k in ("x", "dt", "z"):
            check("d" + k, g[k][B - 1:, :, cs], ref[k], tol[k])
        for k in ("B", "C"):
            check("d" + k, g[k][B - 1:, :, grp:grp + 1], ref[k], tol[k])
        for k in ("A", "D", "dt_bias"):
            check("d" + k, g[k][cs], ref[k], tol[k])
        check("dstate", g["state"][B - 1:, cs], ref["state"], tol["state"])
    assert bool((g["x"][:3] == 0).all()) and bool((g["x"][B - 2] == 0).all())


def test_scan_of_one_long_sequence():
    """Rates of 1 and more and steps of 1 and more: after 200 tokens a state is forgotten to e^-200, so that the
    last tokens are those of the oracle started 300 before the end."""
    from linear_rnn_sequence_wkv7_amd import ssm
    L, N, tail, cs = B * T, 16, 300, slice(C - 20, C)
    x, z = normal(1, 1, L, C), normal(2, 1, L, C)
    dt = normal(3, 1, L, C).abs_().add_(1)
    Bm, Cm = normal(4, 1, L, 1, N), normal(5, 1, L, 1, N)
    A = -(1 + np.random.default_rng(0).random((C, N))).astype(np.float32)
    _, D, _ = parameters(N)
    a, kw = (x, dt, to_dev(A), Bm, Cm), dict(D=to_dev(D), z=z, softplus=False)
    y, s = ssm.ssm_forward(*a, **kw)
    p = {"x": host(x[:, -tail:, cs]), "dt": host(dt[:, -tail:, cs]), "z": host(z[:, -tail:, cs]), "Bm": host(Bm[:, -tail:]), "Cm": host(Cm[:, -tail:]),
         "A": A[cs], "D": D[cs], "dt_bias": None, "state": None}
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(p, tail, None, False)
    check("y", y[:, -100:, cs], y_ref[:, -100:], y_tol[:, -100:])
    check("state", s[:, cs], s_ref, s_tol)
    dy = normal(6, 1, L, C)
    g = ssm.ssm_backward(*a, dy, **kw)
    torch().cuda.synchronize()
    ref, tol = S.scan_bounds(p, tail, None, False, dy=host(dy[:, -tail:, cs]))
    for k in ("x", "dt", "z"):
        check("d" + k, g[k][:, -100:, cs], ref[k][:, -100:], tol[k][:, -100:])


def test_scan_step_on_a_large_pool():
    from linear_rnn_sequence_wkv7_amd import ssm
    Sp, N, rows = 32800, 16, [32799, 0, 5, 32768]
    st = normal(1, Sp, C, N, dtype="f32")
    assert st.numel() > 1 << 31
    x = S.scan_inputs(3, len(rows), 1, C, N, 1, "f32", step=True)
    old = host(st[rows])
    d = {k: to_dev(v) for k, v in x.items()}
    y = ssm.ssm_step(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], st, D=d["D"], dt_bias=d["dt_bias"], z=d["z"],
                     state_index=torch().tensor(rows, dtype=torch().int32, device="cuda"))
    torch().cuda.synchronize()
    one = {k: v[:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in x.items()}
    one["state"] = old
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(one, 1, None, True)
    check("y", y, y_ref[:, 0], y_tol[:, 0])
    check("state", st[rows], s_ref, s_tol)


@pytest.mark.parametrize("Bc,Tc", [(B, T), (1, B * T)])
def test_convolution(Bc, Tc):
    from linear_rnn_sequence_wkv7_amd import shortconv
    K, tail = 4, min(Tc, 300)
    rng = np.random.default_rng(2)
    w, bias = rng.standard_normal((C, K)).astype(np.float32), rng.standard_normal(C).astype(np.float32)
    x, state = normal(1, Bc, Tc, C), normal(2, Bc, K - 1, C)
    y, s = shortconv.shortconv_forward(x, to_dev(w), bias=to_dev(bias), state=state)
    dy = torch().zeros(Bc, Tc, C, device="cuda", dtype=torch().bfloat16)
    dy[-1, -tail:] = normal(3, tail, C)
    ds = normal(4, Bc, K - 1, C, dtype="f32")
    g = shortconv.shortconv_backward(x, to_dev(w), dy, bias=to_dev(bias), state=state, dstate=ds)
    torch().cuda.synchronize()
    before = host(state[-1:] if tail == Tc else x[-1:, -tail - K + 1:-tail])   # the inputs before the tail
    args = (host(x[-1:, -tail:]), w, bias, before, None, True)
    (y_ref, s_ref), (y_tol, _) = S.conv_bounds(*args)
    check("y", y[-1:, -tail:], y_ref, y_tol)
    np.testing.assert_array_equal(to_host(s[-1:].contiguous()), s_ref)
    ref, tol = S.conv_bounds(*args, host(dy[-1:, -tail:]), host(ds[-1:]))
    check("dx", g["x"][-1:, -tail:], ref["x"], tol["x"])
    # the sums over all the tokens: everything before the tail adds 0
    for k in ("w", "bias"):
        check("d" + k, g[k], ref[k], tol[k])
    if Bc > 1:
        check("dstate", g["state"][-1:], ref["state"], tol["state"])


def test_convolution_step_on_a_large_pool():
    from linear_rnn_sequence_wkv7_amd import shortconv
    Sp, K, rows = 175000, 4, [174999, 0, 7, 174763]
    st = normal(1, Sp, K - 1, C)
    assert st.numel() > 1 << 31
    rng = np.random.default_rng(5)
    w, bias = rng.standard_normal((C, K)).astype(np.float32), rng.standard_normal(C).astype(np.float32)
    x, old = normal(2, len(rows), C), host(st[rows])
    y = shortconv.shortconv_step(x, to_dev(w), st, bias=to_dev(bias), state_index=torch().tensor(rows, dtype=torch().int32, device="cuda"))
    torch().cuda.synchronize()
    (y_ref, s_ref), (y_tol, _) = S.conv_bounds(host(x[:, None]), w, bias, old, None, True)
    check("y", y, y_ref[:, 0], y_tol[:, 0])
    np.testing.assert_array_equal(to_host(st[rows]), s_ref)


@pytest.mark.parametrize("Bn,Tn,Cn,G", [(B * T, 1, C, 64), (B * T, 1, 4128, 43), (B, T, C, 64), (4, B * T // 4, C, 64), (B * T, 1, C, 1)],
                         ids=["rows", "waves", "registers", "partial_sums", "whole_rows"])
def test_norm(Bn, Tn, Cn, G):
    """The last group of the last sequence."""
    from linear_rnn_sequence_wkv7_amd import groupnorm
    rng = np.random.default_rng(G)
    weight, bias = (1 + 0.3 * rng.standard_normal(Cn)).astype(np.float32), (0.3 * rng.standard_normal(Cn)).astype(np.float32)
    x, gate = normal(1, Bn, Tn, Cn), normal(2, Bn, Tn, Cn)
    kw = dict(weight=to_dev(weight), bias=to_dev(bias), gate=gate, act="silu")
    y, mean, rstd = groupnorm.groupnorm_forward(x, G, **kw)
    dy = torch().zeros(Bn, Tn, Cn, device="cuda", dtype=torch().bfloat16)
    dy[-1] = normal(3, Tn, Cn)
    g = groupnorm.groupnorm_backward(x, G, dy, mean, rstd, **kw)
    torch().cuda.synchronize()
    cs = slice(Cn - Cn // G, Cn)
    args = (host(x[-1:, :, cs]), 1, weight[cs], bias[cs], host(gate[-1:, :, cs]), True, 1e-5, None)
    (y_ref, m_ref, r_ref), (y_tol, m_tol, r_tol) = S.norm_bounds(*args)
    check("y", y[-1:, :, cs], y_ref, y_tol)
    check("mean", mean[-1:, -1:], m_ref, m_tol)
    check("rstd", rstd[-1:, -1:], r_ref, r_tol)
    ref, tol = S.norm_bounds(*args, dy=host(dy[-1:, :, cs]))
    check("dx", g["x"][-1:, :, cs], ref["x"], tol["x"])
    check("dgate", g["gate"][-1:, :, cs], ref["gate"], tol["gate"])
    check("dweight", g["weight"][cs], ref["weight"], tol["weight"])
    check("dbias", g["bias"][cs], ref["bias"], tol["bias"])
    assert bool((g["x"][0] == 0).all())
