"""GPU parity of the selective state space scan against the fp64 oracle, its
gradients, its single-token form, and what a caller may do with them."""
import numpy as np
import pytest

from oracle import seq_oracle as O
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
    from linear_rnn_sequence_wkv7_amd import ssm
    return ssm


def dev_args(x):
    d = {k: to_dev(v) for k, v in x.items()}
    return (d["x"], d["dt"], d["A"], d["Bm"], d["Cm"]), dict(D=d["D"], dt_bias=d["dt_bias"], z=d["z"])


def lens(lengths):
    return None if lengths is None else torch().tensor(lengths, dtype=torch().int32, device="cuda")


CASES = [
    # B, T, C, N, G, dtype, lengths, z, state
    (1, 1, 1, 1, 1, "f32", None, False, False),
    (2, 3, 5, 3, 1, "bf16", None, True, True),
    (1, 15, 16, 16, 1, "f32", None, True, False),
    (1, 16, 17, 16, 1, "bf16", None, True, True),
    (2, 17, 64, 16, 2, "f32", [17, 5], True, True),
    (3, 63, 40, 8, 4, "bf16", [1, 0, 63], True, True),
    (1, 64, 33, 12, 1, "f32", None, False, True),
    (2, 65, 24, 16, 3, "bf16", [64, 65], True, False),
    (1, 127, 20, 5, 1, "f32", None, True, True),
    (2, 129, 36, 16, 1, "f32", [129, 66], True, True),
    (1, 300, 20, 32, 2, "bf16", None, True, True),
    (2, 130, 9, 20, 1, "f32", [7, 130], True, True),
    (1, 200, 13, 64, 1, "f32", None, True, True),
    (2, 70, 10, 33, 5, "bf16", [70, 69], True, True),
    (2, 50, 20, 24, 1, "f32", [50, 9], True, True),      # rows of lanes without states
    (1, 50, 20, 24, 2, "bf16", None, True, True),
    (2, 50, 20, 48, 1, "f32", None, True, True),
    (1, 50, 20, 48, 2, "bf16", None, True, True),
    (1, 50, 20, 40, 1, "f32", None, True, True),
    (600, 33, 16, 16, 1, "bf16", None, True, False),     # many sequences: fewer waves over the tokens
    (70, 40, 520, 4, 1, "f32", None, False, True),
    (3, 50, 0, 16, 1, "f32", None, True, True),
    (0, 50, 8, 16, 1, "f32", None, True, True),
]
IDS = ["B{}_T{}_C{}_N{}_G{}_{}".format(*c[:6]) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("softplus", [True, False])
def test_forward(case, softplus):
    B, T, C, N, G, dtype, lengths, z, state = case
    x = S.scan_inputs(T * 7 + C, B, T, C, N, G, dtype, z=z, state=state, D=z, bias=True)
    if not softplus:   # the steps are given: positive ones
        x["dt"] = S.as_dtype(np.abs(O.as_f64(x["dt"])) * 0.3, dtype)
        x["dt_bias"] = None
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, T, lengths, softplus, B=B, Cg=C // G)
    a, kw = dev_args(x)
    y_dtype = "f32" if T % 2 else None
    y, s = M().ssm_forward(*a, **kw, state=to_dev(x["state"]), lengths=lens(lengths), softplus=softplus, y_dtype=y_dtype)
    torch().cuda.synchronize()
    S.check("y", to_host(y), y_ref, y_tol, bf16=y.dtype == torch().bfloat16)
    S.check("state", to_host(s), s_ref, s_tol)


@pytest.mark.parametrize("case", [c for c in CASES if c[0] * c[2] < 30000], ids=[i for i, c in zip(IDS, CASES) if c[0] * c[2] < 30000])
@pytest.mark.parametrize("kept", [True, False])
def test_backward(case, kept):
    B, T, C, N, G, dtype, lengths, z, state = case
    x = S.scan_inputs(T * 11 + C, B, T, C, N, G, dtype, z=z, state=state, D=z)
    rng = np.random.default_rng(T)
    dy = S.as_dtype(rng.standard_normal((B, T, C)), dtype)
    ds = rng.standard_normal((B, C, N)).astype(np.float32) if state else None
    ref, tol = S.scan_bounds(x, T, lengths, True, dy=dy, dstate=ds, B=B, Cg=C // G)
    a, kw = dev_args(x)
    kw.update(state=to_dev(x["state"]), lengths=lens(lengths))
    saved = None
    if kept:
        saved = torch().empty(M().ssm_checkpoint_bytes(B, T, C, N), dtype=torch().uint8, device="cuda")
        M().ssm_forward(*a, **kw, checkpoints=saved)
    g = M().ssm_backward(*a, to_dev(dy), dstate=to_dev(ds), checkpoints=saved, **kw)
    torch().cuda.synchronize()
    for k in ref:
        if g[k] is None:
            assert k in ("z", "D") and not z
            continue
        S.check("d" + k, to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == torch().bfloat16)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", range(1, 65))
def test_every_number_of_states(N, dtype):
    """Forward, gradients and a step, with channels and groups of odd and even sizes."""
    G, Cg = (1, 17) if N % 3 == 0 else (2, 10) if N % 3 == 1 else (3, 18)
    B, T, C = 2, 37 + N % 3 * 16, G * Cg
    x = S.scan_inputs(N, B, T, C, N, G, dtype, state=True)
    lengths = [T, T // 2]
    dy = S.as_dtype(np.random.default_rng(N).standard_normal((B, T, C)), dtype)
    a, kw = dev_args(x)
    kw.update(state=to_dev(x["state"]), lengths=lens(lengths))
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, T, lengths, True, B=B, Cg=Cg)
    y, s = M().ssm_forward(*a, **kw)
    S.check("y", to_host(y), y_ref, y_tol, bf16=dtype == "bf16")
    S.check("state", to_host(s), s_ref, s_tol)
    ref, tol = S.scan_bounds(x, T, lengths, True, dy=dy, B=B, Cg=Cg)
    g = M().ssm_backward(*a, to_dev(dy), **kw)
    for k in ref:
        S.check("d" + k, to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == torch().bfloat16)
    first = {k: None if v is None else v[:, :1] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in x.items()}
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(first, 1, None, True, B=B, Cg=Cg)
    one = lambda t: t[:, 0].contiguous()
    st = to_dev(x["state"])
    y = M().ssm_step(one(a[0]), one(a[1]), a[2], one(a[3]), one(a[4]), st, D=kw["D"], dt_bias=kw["dt_bias"], z=one(kw["z"]))
    S.check("step y", to_host(y), y_ref[:, 0], y_tol[:, 0], bf16=dtype == "bf16")
    S.check("step state", to_host(st), s_ref, s_tol)


def test_gradient_against_differences():
    """The gradient along a direction against the forward's own central difference.  In fp32 a
    step of 2^-6 is off by its square (times the third derivative) and by the loss' rounding
    over the step: 1e-3 of the sum of the terms' sizes covers both."""
    B, T, C, N = 1, 70, 16, 16
    x = S.scan_inputs(5, B, T, C, N, dtype="f32", state=True)
    rng = np.random.default_rng(6)
    dy, ds = rng.standard_normal((B, T, C)).astype(np.float32), rng.standard_normal((B, C, N)).astype(np.float32)
    a, kw = dev_args(x)
    g = M().ssm_backward(*a, to_dev(dy), dstate=to_dev(ds), state=to_dev(x["state"]), **kw)
    key = dict(x="x", dt="dt", A="A", Bm="B", Cm="C", D="D", dt_bias="dt_bias", z="z", state="state")
    for name, gk in key.items():
        v = rng.standard_normal(x[name].shape).astype(np.float32) * (0.1 if name == "A" else 1.0)
        vals = []
        for sign in (1, -1):
            m = dict(x)
            m[name] = (x[name] + sign * np.float32(2.0 ** -6) * v).astype(np.float32)
            am, km = dev_args(m)
            y, s = M().ssm_forward(*am, state=to_dev(m["state"]), **km)
            vals.append((to_host(y) * dy).sum() + (to_host(s) * ds).sum())
        num = (vals[0] - vals[1]) / 2.0 ** -5
        gv = to_host(g[gk]) * v
        assert abs(num - gv.sum()) <= 1e-3 * np.abs(gv).sum() + 1e-3 * np.abs(dy).sum() / 64, name


def test_padding_values_do_not_matter():
    """NaN and infinities behind a sequence's end reach neither y nor state nor any gradient."""
    B, T, C, N, G = 2, 80, 24, 16, 2
    lengths = [37, 0]
    x = S.scan_inputs(9, B, T, C, N, G, "f32", state=True)
    clean = {k: None if v is None else v.copy() for k, v in x.items()}
    for k in ("x", "dt", "Bm", "Cm", "z"):
        for b, n in enumerate(lengths):
            x[k][b, n:] = np.nan if k != "dt" else np.inf
            clean[k][b, n:] = 0
    dy = np.random.default_rng(1).standard_normal((B, T, C)).astype(np.float32)
    out = []
    for m, d in ((x, dy.copy()), (clean, dy.copy())):
        for b, n in enumerate(lengths):
            d[b, n:] = np.nan if m is x else 0
        a, kw = dev_args(m)
        kw.update(state=to_dev(m["state"]), lengths=lens(lengths))
        y, s = M().ssm_forward(*a, **kw)
        g = M().ssm_backward(*a, to_dev(d), **kw)
        torch().cuda.synchronize()
        out.append({"y": to_host(y), "s": to_host(s), **{k: to_host(v) for k, v in g.items()}})
    for k in out[0]:
        np.testing.assert_array_equal(out[0][k], out[1][k], err_msg=k)
    assert np.all(out[0]["y"][1] == 0) and np.all(out[0]["x"][0, 37:] == 0)
    np.testing.assert_array_equal(out[0]["s"][1], x["state"][1])


def test_no_tokens():
    """T = 0: the state goes over, its gradient back, and the parameters have none."""
    t = torch()
    B, C, N = 2, 20, 16
    x = S.scan_inputs(1, B, 0, C, N, dtype="bf16", state=True)
    a, kw = dev_args(x)
    st = to_dev(x["state"])
    y, s = M().ssm_forward(*a, state=st, **kw)
    assert y.shape == (B, 0, C) and t.equal(s, st)
    _, s = M().ssm_forward(*a, **kw)
    assert bool((s == 0).all())
    ds = t.randn(B, C, N, device="cuda")
    g = M().ssm_backward(*a, y, dstate=ds, state=st, **kw)
    assert t.equal(g["state"], ds)
    assert all(bool((g[k] == 0).all()) for k in ("A", "D", "dt_bias"))


@pytest.mark.parametrize("B,C,N,dtype", [(2, 20, 16, "bf16"), (3, 7, 5, "f32"), (700, 600, 16, "f32")])
def test_gradients_without_tokens_need_no_workspace(B, C, N, dtype):
    """T = 0, with and without a gradient of the state, into outputs that held something."""
    t = torch()
    x = S.scan_inputs(2, B, 0, C, N, dtype=dtype)
    a, kw = dev_args(x)
    ds = t.randn(B, C, N, device="cuda")
    full = lambda *s: t.full(s, 7.0, device="cuda")
    assert M().ssm_backward_workspace_bytes(B, 0, C, N) == M().ssm_backward_workspace_bytes(B, 0, C, N, checkpoints=False) == 0
    for given in (ds, None):
        grads = {"A": full(C, N), "D": full(C), "dt_bias": full(C), "state": full(B, C, N)}
        g = M().ssm_backward(*a, a[0], dstate=given, grads=grads, **kw)
        assert all(g[k] is grads[k] for k in grads)
        assert t.equal(g["state"], ds if given is not None else t.zeros_like(ds))
        assert all(bool((g[k] == 0).all()) for k in ("A", "D", "dt_bias"))


def test_lengths_from_the_middle_of_a_tensor():
    t = torch()
    x = S.scan_inputs(3, 2, 20, 8, 16, dtype="f32")
    a, kw = dev_args(x)
    y1, s1 = M().ssm_forward(*a, **kw, lengths=t.tensor([99, 7, 20], dtype=t.int32, device="cuda")[1:])
    y2, s2 = M().ssm_forward(*a, **kw, lengths=lens([7, 20]))
    assert t.equal(y1, y2) and t.equal(s1, s2)


def test_lengths_out_of_range_are_held():
    x = S.scan_inputs(3, 2, 20, 8, 16, dtype="f32")
    a, kw = dev_args(x)
    y1, s1 = M().ssm_forward(*a, **kw, lengths=lens([-5, 99]))
    y2, s2 = M().ssm_forward(*a, **kw, lengths=lens([0, 20]))
    assert torch().equal(y1, y2) and torch().equal(s1, s2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,N,G", [(64, 16, 1), (37, 16, 1), (24, 5, 3), (10, 64, 1), (8, 33, 2), (70, 2, 1)])
def test_step(C, N, G, dtype):
    """Single tokens against the oracle, on a pool: rows in no order, rows without a request, a row
    that names a state again."""
    B, Sp = 7, 9
    x = S.scan_inputs(C + N, B, 1, C, N, G, dtype, step=True)
    rng = np.random.default_rng(C)
    pool = rng.standard_normal((Sp, C, N)).astype(np.float32)
    index = [4, -1, 0, 8, 4, 9, 2]
    a, kw = dev_args(x)
    st = to_dev(pool)
    y = M().ssm_step(*a, st, state_index=torch().tensor(index, dtype=torch().int32, device="cuda"), **kw)
    torch().cuda.synchronize()
    rows = [0, 2, 3, 6]
    pick = {k: (v[rows][:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in x.items()}
    pick["state"] = pool[[index[r] for r in rows]]
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(pick, 1, None, True)
    S.check("y", to_host(y)[rows], y_ref[:, 0], y_tol[:, 0], bf16=dtype == "bf16")
    new = to_host(st)
    S.check("state", new[[index[r] for r in rows]], s_ref, s_tol)
    assert np.all(to_host(y)[[1, 4, 5]] == 0)
    np.testing.assert_array_equal(new[[1, 3, 5, 6, 7]], pool[[1, 3, 5, 6, 7]])


def test_steps_follow_the_prompt():
    """A prompt, then its next tokens one by one, is the longer prompt: to the bounds of both, with
    the states' own."""
    B, T, C, N = 3, 41, 48, 16
    x = S.scan_inputs(8, B, T, C, N, dtype="f32")
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, T, None, True, B=B, Cg=C)
    a, kw = dev_args(x)
    cut = lambda t0, t1: (tuple(v[:, t0:t1].contiguous() if v.dim() >= 3 else v for v in a),
                          {k: v[:, t0:t1].contiguous() if v.dim() == 3 else v for k, v in kw.items()})
    a0, k0 = cut(0, 30)
    y, s = M().ssm_forward(*a0, **k0)
    S.check("y", to_host(y), y_ref[:, :30], y_tol[:, :30])
    for t in range(30, T):
        a1, k1 = cut(t, t + 1)
        a1 = tuple(v[:, 0] if v.dim() >= 3 else v for v in a1)
        k1 = {k: v[:, 0] if v.dim() == 3 else v for k, v in k1.items()}
        y1 = M().ssm_step(*a1, s, **k1)
        S.check(f"y {t}", to_host(y1), y_ref[:, t], y_tol[:, t])
    S.check("state", to_host(s), s_ref, s_tol)


def test_many_rows_share_an_index():
    """More rows than a workgroup has threads, every state named several times."""
    B, C, N, Sp = 700, 16, 16, 50
    x = S.scan_inputs(2, B, 1, C, N, 1, "f32", step=True)
    rng = np.random.default_rng(3)
    pool = rng.standard_normal((Sp, C, N)).astype(np.float32)
    index = rng.integers(-2, Sp + 2, B).astype(np.int32)
    first = [b for b in range(B) if 0 <= index[b] < Sp and index[b] not in index[:b]]
    a, kw = dev_args(x)
    st = to_dev(pool)
    y = to_host(M().ssm_step(*a, st, state_index=to_dev(index), **kw))
    pick = {k: (v[first][:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in x.items()}
    pick["state"] = pool[index[first]]
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(pick, 1, None, True)
    S.check("y", y[first], y_ref[:, 0], y_tol[:, 0])
    S.check("state", to_host(st)[index[first]], s_ref, s_tol)
    others = np.setdiff1d(np.arange(B), first)
    assert np.all(y[others] == 0)


def test_in_place_state_and_repeatability():
    x = S.scan_inputs(4, 2, 100, 40, 16, dtype="bf16", state=True)
    a, kw = dev_args(x)
    y1, s1 = M().ssm_forward(*a, **kw, state=to_dev(x["state"]))
    st = to_dev(x["state"])
    y2, s2 = M().ssm_forward(*a, **kw, state=st, state_out=st)
    assert s2 is st and torch().equal(s1, s2) and torch().equal(y1, y2)
    dy = to_dev(S.as_dtype(np.random.default_rng(0).standard_normal((2, 100, 40)), "bf16"))
    g1 = M().ssm_backward(*a, dy, **kw)
    g2 = M().ssm_backward(*a, dy, **kw)
    for k in g1:
        assert torch().equal(g1[k], g2[k]), k


@pytest.mark.parametrize("T,C,lens_", [(500, 48, None), (1000, 32, [1000, 777])])
def test_long_sequences_in_rounds(T, C, lens_):
    """Several rounds of the kernels, each taking up where the other left (also the checkpoints), for
    every number of runs: few channels here, many sequences below."""
    x = S.scan_inputs(T, 2, T, C, 16, dtype="f32", state=True)
    dy = np.random.default_rng(T).standard_normal((2, T, C)).astype(np.float32)
    a, kw = dev_args(x)
    kw.update(state=to_dev(x["state"]), lengths=lens(lens_))
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, T, lens_, True, B=2, Cg=C)
    saved = torch().empty(M().ssm_checkpoint_bytes(2, T, C, 16), dtype=torch().uint8, device="cuda")
    y, s = M().ssm_forward(*a, **kw, checkpoints=saved)
    S.check("y", to_host(y), y_ref, y_tol)
    S.check("state", to_host(s), s_ref, s_tol)
    ref, tol = S.scan_bounds(x, T, lens_, True, dy=dy, B=2, Cg=C)
    g = M().ssm_backward(*a, to_dev(dy), checkpoints=saved, **kw)
    for k in ref:
        S.check("d" + k, to_host(g[k]), ref[k], tol[k])
    # the same two sequences among many: other numbers of runs
    for copies in (100, 600):
        rep = lambda v: v.repeat(copies, *([1] * (v.dim() - 1)))
        am = tuple(rep(v) if v.dim() >= 3 else v for v in a)
        km = {k: rep(v) if v is not None and (v.dim() == 3 or k == "lengths") else v for k, v in kw.items()}
        ym, sm = M().ssm_forward(*am, **km)
        S.check("y", to_host(ym[-2:]), y_ref, y_tol)
        S.check("state", to_host(sm[-2:]), s_ref, s_tol)


@pytest.mark.parametrize("N,T,copies", [(16, 300, 1), (16, 40, 200), (16, 40, 600), (16, 40, 1100), (8, 300, 1), (8, 40, 200), (32, 40, 1),
                                        (32, 40, 150), (32, 40, 300), (64, 40, 1), (64, 40, 150), (15, 300, 1)])
def test_gradients_of_many_sequences(N, T, copies):
    """Two sequences, many times: every number of runs that the backward takes.  The parameters' gradients are the
    copies' sums, within the bound for so large a batch."""
    x = S.scan_inputs(N + copies, 2, T, 16, N, dtype="f32", state=True)
    rng = np.random.default_rng(copies)
    dy, ds = rng.standard_normal((2, T, 16)).astype(np.float32), rng.standard_normal((2, 16, N)).astype(np.float32)
    ref, tol = S.scan_bounds(x, T, None, True, dy=dy, dstate=ds, B=2, Cg=16)
    tol_all = S.scan_bounds(x, T, None, True, dy=dy, dstate=ds, B=2 * copies, Cg=16)[1]
    rep = lambda v: v.repeat(copies, *([1] * (v.dim() - 1)))
    a, kw = dev_args(x)
    a = tuple(rep(v) if v.dim() >= 3 else v for v in a)
    kw = {k: rep(v) if v is not None and v.dim() == 3 else v for k, v in kw.items()}
    g = M().ssm_backward(*a, rep(to_dev(dy)), dstate=rep(to_dev(ds)), state=rep(to_dev(x["state"])), **kw)
    for k in ref:
        if k in ("A", "D", "dt_bias"):
            S.check("d" + k, to_host(g[k]), copies * ref[k], copies * tol_all[k])
        else:
            S.check("d" + k, to_host(g[k][-2:]), ref[k], tol[k])
            assert torch().equal(g[k][:2], g[k][-2:])


def test_step_sizes_at_the_ends():
    """softplus far below zero keeps its relative accuracy, far above it is the identity; steps
    so long that a decay is 0 leave the newest token only."""
    C, N = 16, 16
    v = np.array([-80, -60, -40, -20, -10, -5, -1, 0, 1, 5, 10, 19, 21, 40, 60, 80], dtype=np.float32)
    x = S.scan_inputs(1, 1, 2, C, N, dtype="f32", z=False, D=False, bias=False)
    x["dt"][:] = v
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, 2, None, True)
    a, kw = dev_args(x)
    y, s = M().ssm_forward(*a, **kw)
    S.check("y", to_host(y), y_ref, y_tol)
    S.check("state", to_host(s), s_ref, s_tol)
    # each channel to its own scale
    assert np.max(np.abs(to_host(s) - s_ref).max(-1) / np.abs(s_ref).max(-1)) <= 600 * S.U


@pytest.mark.parametrize("T,C,N,softplus", [(17, 16, 16, True), (150, 20, 16, True), (150, 20, 24, True), (70, 18, 7, False)])
def test_growing_states(T, C, N, softplus):
    """Rates of both signs, 0 among them, and given steps of both signs: states that grow up to some e^10."""
    B = 2
    x = S.scan_inputs(T, B, T, C, N, 1, "f32", state=True, bias=softplus)
    rng = np.random.default_rng(N)
    x["A"] = rng.uniform(-0.5, 0.1, (C, N)).astype(np.float32)
    x["A"][0], x["A"][1, 0] = 0.0, 0.1
    if not softplus:
        x["dt"] = (rng.standard_normal((B, T, C)) * 0.4).astype(np.float32)
    dy, ds = rng.standard_normal((B, T, C)).astype(np.float32), rng.standard_normal((B, C, N)).astype(np.float32)
    a, kw = dev_args(x)
    kw["state"] = to_dev(x["state"])
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, T, None, softplus, B=B, Cg=C)
    y, s = M().ssm_forward(*a, softplus=softplus, **kw)
    S.check("y", to_host(y), y_ref, y_tol)
    S.check("state", to_host(s), s_ref, s_tol)
    ref, tol = S.scan_bounds(x, T, None, softplus, dy=dy, dstate=ds, B=B, Cg=C)
    g = M().ssm_backward(*a, to_dev(dy), dstate=to_dev(ds), softplus=softplus, **kw)
    torch().cuda.synchronize()
    for k in ref:
        if g[k] is not None:
            S.check("d" + k, to_host(g[k]), ref[k], tol[k])
