"""What a caller hands in as outputs and workspace: every element of an output is written,
whatever it held (NaN here), nothing beside it, and nothing of the workspace is taken for
more than scratch (all its bits are set here).  Inputs stand between NaN, which no result
shows.  Results equal those of the call that allocates its own, bit for bit."""
import numpy as np
import pytest

from tests import seq_util as S
from tests.gpu_util import announce, to_dev, torch

pytestmark = pytest.mark.gpu

GUARD = 4096   # elements on each side


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


class Guarded:
    """Tensors inside larger ones of NaN (integers: of a large negative number)."""

    def __init__(self):
        self.all = []

    def out(self, like, dtype=None):
        t = torch()
        dtype = like.dtype if dtype is None else dtype
        whole = t.full((like.numel() + 2 * GUARD,), float("nan") if dtype.is_floating_point else -77777, dtype=dtype, device="cuda")
        self.all.append(whole)
        return whole[GUARD:GUARD + like.numel()].view(like.shape)

    def put(self, v):
        """A copy of v between guards."""
        if v is None:
            return None
        g = self.out(v)
        g.copy_(v)
        return g

    def check(self):
        for w in self.all:
            for part in (w[:GUARD], w[-GUARD:]):
                assert bool(part.isnan().all() if w.dtype.is_floating_point else (part == -77777).all())


def scratch(n):
    """n bytes of ones between others; the second value checks those."""
    t = torch()
    whole = t.full((n + 8192,), 255, dtype=t.uint8, device="cuda")
    return whole[4096:4096 + n], lambda: bool((whole[:4096] == 255).all() and (whole[4096 + n:] == 255).all())


def same(what, got, want):
    t = torch()
    assert got.dtype == want.dtype and t.equal(got, want), f"{what}: {int((got != want).sum())} of {want.numel()} differ"


def lens(lengths):
    return None if lengths is None else torch().tensor(lengths, dtype=torch().int32, device="cuda")


SCANS = [
    # B, T, C, N, G, dtype, lengths
    (3, 15, 21, 16, 1, "f32", [15, 0, 7]),
    (3, 40, 37, 5, 1, "bf16", [33, 0, 17]),
    (2, 65, 36, 16, 3, "bf16", [64, 1]),
    (2, 150, 36, 12, 2, "f32", [150, 31]),
    (2, 300, 32, 16, 2, "bf16", [299, 129]),
    (3, 70, 20, 24, 1, "f32", [70, 0, 33]),
    (2, 70, 14, 40, 7, "bf16", [69, 32]),
    (700, 33, 18, 16, 1, "f32", None),
    (300, 100, 32, 7, 2, "bf16", None),
    (2100, 20, 16, 16, 1, "bf16", None),
]


@pytest.mark.parametrize("case", SCANS, ids=["B{}_T{}_C{}_N{}_G{}_{}".format(*c[:6]) for c in SCANS])
def test_scan(case):
    from linear_rnn_sequence_wkv7_amd import ssm
    t = torch()
    B, T, C, N, G, dtype, lengths = case
    x = {k: to_dev(v) for k, v in S.scan_inputs(T + C, B, T, C, N, G, dtype, state=True).items()}
    dy, ds = t.randn(B, T, C, device="cuda").to(x["x"].dtype), t.randn(B, C, N, device="cuda")
    names = ("x", "dt", "A", "Bm", "Cm")

    def calls(x, dy, ds, ln, out=None, ws=None, ck=None):
        o = out or {}
        kw = dict(D=x["D"], dt_bias=x["dt_bias"], z=x["z"], state=x["state"], lengths=ln)
        y, s = ssm.ssm_forward(*(x[k] for k in names), **kw, y=o.get("y"), state_out=o.get("s"), checkpoints=ck)
        g = ssm.ssm_backward(*(x[k] for k in names), dy, dstate=ds, checkpoints=ck, workspace=ws, **kw,
                             grads=o.get("g"))
        return y, s, g
    for kept in (False, True):
        nck = ssm.ssm_checkpoint_bytes(B, T, C, N)
        ck = t.empty(nck, dtype=t.uint8, device="cuda") if kept else None
        y, s, g = calls(x, dy, ds, lens(lengths), ck=ck)
        q = Guarded()
        ws, ws_ok = scratch(ssm.ssm_backward_workspace_bytes(B, T, C, N, G=G, checkpoints=kept))
        ck2, ck_ok = scratch(nck)
        out = {"y": q.out(y), "s": q.out(s), "g": {k: q.out(v) for k, v in g.items()}}
        y2, s2, g2 = calls({k: q.put(v) for k, v in x.items()}, q.put(dy), q.put(ds), q.put(lens(lengths)), out, ws, ck2 if kept else None)
        t.cuda.synchronize()
        assert y2 is out["y"] and s2 is out["s"] and all(g2[k] is out["g"][k] for k in g2)
        same("y", y2, y)
        same("state", s2, s)
        for k in g:
            same("d" + k, g2[k], g[k])
        if kept:
            same("checkpoints", ck2, ck)
        q.check()
        assert ws_ok() and ck_ok()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,K,lengths", [(3, 7, 5, 4, [7, 0, 2]), (2, 33, 24, 3, [33, 31]), (3, 70, 18, 2, [69, 0, 70]), (2, 300, 72, 4, None),
                                             (40, 100, 516, 4, None)])
def test_convolution(B, T, C, K, lengths, dtype):
    from linear_rnn_sequence_wkv7_amd import shortconv
    t = torch()
    dt = t.float32 if dtype == "f32" else t.bfloat16
    r = lambda *s: t.randn(*s, device="cuda")
    x, state, dy, ds, w, bias = r(B, T, C).to(dt), r(B, K - 1, C).to(dt), r(B, T, C).to(dt), r(B, K - 1, C), r(C, K), r(C)

    def calls(x, w, bias, state, dy, ds, ln, o=None, ws=None):
        o = o or {}
        kw = dict(bias=bias, state=state, lengths=ln)
        y, s = shortconv.shortconv_forward(x, w, **kw, y=o.get("y"), state_out=o.get("s"))
        return y, s, shortconv.shortconv_backward(x, w, dy, dstate=ds, workspace=ws, grads=o.get("g"), **kw)
    y, s, g = calls(x, w, bias, state, dy, ds, lens(lengths))
    q = Guarded()
    ws, ws_ok = scratch(shortconv.shortconv_backward_workspace_bytes(B, T, C, K))
    out = {"y": q.out(y), "s": q.out(s), "g": {k: q.out(v) for k, v in g.items()}}
    y2, s2, g2 = calls(*(q.put(v) for v in (x, w, bias, state, dy, ds, lens(lengths))), out, ws)
    t.cuda.synchronize()
    same("y", y2, y)
    same("state", s2, s)
    for k in g:
        assert g2[k] is out["g"][k]
        same("d" + k, g2[k], g[k])
    q.check()
    assert ws_ok()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,G,lengths", [(5, 1, 128, 4, None), (300, 1, 1040, 65, None), (3, 1, 96, 1, [1, 0, 1]), (4, 1, 1599, 1, None), (7, 1, 21, 3, None),
                                             (2, 1, 4100, 1, None), (3, 40, 48, 2, [40, 7, 0]), (2, 33, 15, 5, None), (2, 1100, 32, 2, [1100, 600]),
                                             (2, 3000, 96, 2, [2999, 30]), (1, 1000, 514, 1, None), (1, 130, 1999, 1, [77]), (1, 3000, 24, 3, None)])
def test_norm(B, T, C, G, lengths, dtype):
    from linear_rnn_sequence_wkv7_amd import groupnorm
    t = torch()
    dt = t.float32 if dtype == "f32" else t.bfloat16
    r = lambda *s: t.randn(*s, device="cuda")
    x, gate, dy, weight, bias = r(B, T, C).to(dt), r(B, T, C).to(dt), r(B, T, C).to(dt), r(C), r(C)

    def calls(x, gate, dy, weight, bias, ln, o=None, ws=None):
        o = o or {}
        kw = dict(weight=weight, bias=bias, gate=gate, act="silu", lengths=ln)
        fw = groupnorm.groupnorm_forward(x, G, y=o.get("y"), mean=o.get("mean"), rstd=o.get("rstd"), workspace=ws, **kw)
        return *fw, groupnorm.groupnorm_backward(x, G, dy, fw[1], fw[2], workspace=ws, grads=o.get("g"), **kw)
    y, mean, rstd, g = calls(x, gate, dy, weight, bias, lens(lengths))
    q = Guarded()
    ws, ws_ok = scratch(max(groupnorm.groupnorm_workspace_bytes(B, T, C, G), groupnorm.groupnorm_backward_workspace_bytes(B, T, C, G)))
    out = {"y": q.out(y), "mean": q.out(mean), "rstd": q.out(rstd), "g": {k: q.out(v) for k, v in g.items()}}
    y2, m2, r2, g2 = calls(*(q.put(v) for v in (x, gate, dy, weight, bias, lens(lengths))), out, ws)
    t.cuda.synchronize()
    same("y", y2, y)
    same("mean", m2, mean)
    same("rstd", r2, rstd)
    for k in g:
        assert g2[k] is out["g"][k]
        same("d" + k, g2[k], g[k])
    q.check()
    assert ws_ok()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,N,G,K", [(3, 21, 16, 1, 4), (7, 36, 5, 3, 3), (1, 64, 64, 2, 2), (1030, 260, 16, 1, 4)])
def test_steps(B, C, N, G, K, dtype):
    """Single tokens on pools between guards; and on a pool without states, where no row has a request."""
    from linear_rnn_sequence_wkv7_amd import shortconv, ssm
    t = torch()
    x = {k: to_dev(v) for k, v in S.scan_inputs(B, B, 1, C, N, G, dtype, step=True).items()}
    index = t.randperm(B + 2, device="cuda")[:B].to(t.int32)
    r = lambda *s: t.randn(*s, device="cuda")
    pool, cpool, w, bias = r(B + 2, C, N), r(B + 2, K - 1, C).to(x["x"].dtype), r(C, K), r(C)

    def calls(x, pool, cpool, w, bias, index, y=None, u=None):
        y = ssm.ssm_step(x["x"], x["dt"], x["A"], x["Bm"], x["Cm"], pool, D=x["D"], dt_bias=x["dt_bias"], z=x["z"], state_index=index, y=y)
        return y, shortconv.shortconv_step(x["x"], w, cpool, bias=bias, state_index=index, y=u)
    a, b = pool.clone(), cpool.clone()
    y, u = calls(x, a, b, w, bias, index)
    q = Guarded()
    a2, b2 = q.put(pool), q.put(cpool)
    y2, u2 = calls({k: q.put(v) for k, v in x.items()}, a2, b2, q.put(w), q.put(bias), q.put(index), q.out(y), q.out(u))
    t.cuda.synchronize()
    for what, got, want in (("y", y2, y), ("state", a2, a), ("u", u2, u), ("inputs", b2, b)):
        same(what, got, want)
    q.check()
    y3, u3 = calls(x, pool[:0], cpool[:0], w, bias, index, q.out(y), q.out(u))
    t.cuda.synchronize()
    assert bool((y3 == 0).all()) and bool((u3 == 0).all())
    q.check()
