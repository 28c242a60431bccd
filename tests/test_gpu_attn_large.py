"""Linear attention and the layer norm on arrays of more than 2^31 elements (more than
2^32 bytes), where every offset of the last rows needs 64 bits: the last sequence, or
the last tokens of a long one, against the oracle."""
import numpy as np
import pytest

from oracle import attn_oracle as O
from tests import attn_util as A
from tests.gpu_util import announce, to_dev, torch
from tests.seq_util import U
from tests.test_gpu_seq_large import check, host, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield
    torch().cuda.empty_cache()


def mod():
    from linear_rnn_sequence_wkv7_amd import linattn
    return linattn


def decays(seed, B, T, H):
    return -0.3 * torch().exp(normal(seed, B, T, H, dtype="f32"))


def test_many_sequences():
    B, T, H, Hk, D = 8200, 64, 64, 32, 64   # the heads' gradients of k, in the workspace, are past 2^32 bytes too
    q, k, v, dy = normal(0, B, T, H, D), normal(1, B, T, Hk, D), normal(2, B, T, H, D), normal(3, B, T, H, D)
    g, st, ds = decays(4, B, T, H), normal(5, B, H, D, D, dtype="f32"), normal(6, B, H, D, D, dtype="f32")
    assert q.numel() > 1 << 31 and st.numel() > 1 << 31
    y, s = mod().linattn_forward(q, k, v, g, scale=0.2, state=st)
    gr = mod().linattn_backward(q, k, v, g, dy, scale=0.2, state=st, dstate=ds)
    torch().cuda.synchronize()
    for b, h in ((B - 1, H - 2), (B - 2, 6), (0, 0)):
        bs, hs, ks = slice(b, b + 1), slice(h, h + 2), slice(h // 2, h // 2 + 1)
        x = {"q": host(q[bs, :, hs]), "k": host(k[bs, :, ks]), "v": host(v[bs, :, hs]), "g": host(g[bs, :, hs]), "state": host(st[bs, hs])}
        (y_ref, s_ref), (y_tol, s_tol) = A.attn_bounds(x, 0.2)
        check("y", y[bs, :, hs], y_ref, y_tol)
        check("state", s[bs, hs], s_ref, s_tol)
        ref, tol = A.attn_grad_bounds(x, host(dy[bs, :, hs]), host(ds[bs, hs]), 0.2)
        for n, got in (("q", gr["q"][bs, :, hs]), ("k", gr["k"][bs, :, ks]), ("v", gr["v"][bs, :, hs]), ("g", gr["g"][bs, :, hs]), ("state", gr["state"][bs, hs])):
            check("d" + n, got, ref[n], tol[n])


def test_one_long_sequence():
    """The state is emptied 150 tokens before the end, so that the oracle needs no more than those."""
    T, H, D, N = 530000, 64, 64, 150
    q, k, v, dy, g = *(normal(i, 1, T, H, D) for i in range(4)), decays(4, 1, T, H)
    assert q.numel() > 1 << 31
    g[:, T - N] = -1e5
    ds = normal(6, 1, H, D, D, dtype="f32")
    y, s = mod().linattn_forward(q, k, v, g, scale=0.2)
    gr = mod().linattn_backward(q, k, v, g, dy, scale=0.2, dstate=ds)
    torch().cuda.synchronize()
    hs, last = slice(H - 2, H), slice(T - N, T)
    part = lambda t: t[:, last, hs]
    x = {**{n: host(part(t)) for n, t in (("q", q), ("k", k), ("v", v), ("g", g))}, "state": None}
    (y_ref, s_ref), (y_tol, s_tol) = A.attn_bounds(x, 0.2)
    check("y", part(y), y_ref, y_tol)
    check("state", s[:, hs], s_ref, s_tol)
    ref, tol = A.attn_grad_bounds(x, host(part(dy)), host(ds[:, hs]), 0.2)
    for n in ("q", "k", "v", "g"):
        check("d" + n, part(gr[n]), ref[n], tol[n])


@pytest.mark.parametrize("D,shared", [(128, 4), (64, 1), (96, 2)])
def test_a_full_chip_repeats(D, shared):
    """Every compute unit with several workgroups for long, which drift apart within a chunk as far as the barriers
    let them: results repeat to the bit, forward and backward, and no row is further from the fp32 kernels' (other
    matrix instructions, chunks of half the length) than y's rounding, 2^-9 of a row's norm, and 2^-16 for each of
    the two operands that y splits in two."""
    t = torch()
    B, T, H = 2, 8192, 32
    q, k, v, dy = (normal(i, B, T, n, D) for i, n in enumerate((H // shared, H // shared, H, H)))
    g = decays(4, B, T, H)
    runs = [(mod().linattn_forward(q, k, v, g, scale=0.1), mod().linattn_backward(q, k, v, g, dy, scale=0.1)) for _ in range(3)]
    wide = [(mod().linattn_forward(q.float(), k.float(), v.float(), g, scale=0.1), mod().linattn_backward(q.float(), k.float(), v.float(), g, dy.float(), scale=0.1))
            for _ in range(2)]
    t.cuda.synchronize()
    for all_runs in (runs, wide):
        (y, st), gr = all_runs[0]
        for (y2, st2), gr2 in all_runs[1:]:
            assert t.equal(y, y2) and t.equal(st, st2)
            for n in gr:
                assert t.equal(gr[n], gr2[n]), n
    for got, want in [(runs[0][0][0], wide[0][0][0])] + [(runs[0][1][n], wide[0][1][n]) for n in "qkv"]:
        off = (got.float() - want).norm(dim=-1) / want.norm(dim=-1)
        assert float(off.max()) < 2.0 ** -8, float(off.max())


def test_step_on_a_large_pool():
    B, S, H, D = 3, 8300, 16, 128
    pool = normal(0, S, H, D, D, dtype="f32")
    assert pool.numel() > 1 << 31
    x = {k: to_dev(v) for k, v in A.attn_inputs(1, B, 1, H, D, D, dtype="bf16", step=True).items() if v is not None}
    rows = [S - 1, 17, S - 2]
    before = host(pool[rows])
    y = mod().linattn_step(*(x[n] for n in "qkvg"), pool, scale=0.1, state_index=torch().tensor(rows, dtype=torch().int32, device="cuda"))
    torch().cuda.synchronize()
    a = [host(x[n]) for n in "qkvg"]
    (ref, s_ref), (mag, s_mag) = (O.attn_step(*a, before, scale=0.1, mag=m) for m in (False, True))
    check("y", y, ref, (2 * D + 20) * U * mag)   # a product, an exponential and two additions for each of 128 terms
    check("pool", pool[rows], s_ref, 8 * U * s_mag)


@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_norm(stream):
    """Only the last sequence's dy is not 0, so that sums over the rows are that sequence's (adding 0 rounds nothing)."""
    from linear_rnn_sequence_wkv7_amd import layernorm
    B, T, C = 8200, 64, 4096
    x, res = normal(0, B, T, C), normal(1, B, T, C, dtype=stream)
    assert x.numel() > 1 << 31
    rng = np.random.default_rng(0)
    w, bias = ((a + 0.2 * rng.standard_normal(C)).astype(np.float32) for a in (1, 0))
    dy = torch().zeros(B, T, C, device="cuda", dtype=torch().bfloat16)
    dy[B - 1] = normal(3, T, C)
    y, h, mean, rstd = layernorm.layernorm_forward(x, residual=res, weight=to_dev(w), bias=to_dev(bias))
    g = layernorm.layernorm_backward(h, dy, mean, rstd, weight=to_dev(w), bias=to_dev(bias), dh=res, x_dtype="bf16")
    torch().cuda.synchronize()
    for b in (B - 1, 0):
        bs = slice(b, b + 1)
        h_ref = A.stream({"x": host(x[bs]), "residual": host(res[bs])})
        assert np.array_equal(host(h[bs]), h_ref)
        (y_ref, m_ref, r_ref), (y_tol, m_tol, r_tol), _ = A.norm_bounds(h_ref, w, bias, 1e-5)
        check("y", y[bs], y_ref, y_tol)
        check("mean", mean[bs], m_ref, m_tol)
        check("rstd", rstd[bs], r_ref, r_tol)
        ref, tol = A.norm_grad_bounds(h_ref, host(dy[bs]), w, host(res[bs]), 1e-5)
        check("dh", g["h"][bs], ref["h"], tol["h"])
        check("dx", g["x"][bs], ref["h"], tol["h"])
        if b == B - 1:
            for n in ("weight", "bias"):
                check("d" + n, g[n], ref[n], tol[n])
