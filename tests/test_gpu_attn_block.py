"""The layer norm, linear attention and the group norm as a layer uses them together:
training and serving chains, captured into HIP graphs, on other streams, with the
caller's outputs and workspaces between guards; and what the bindings refuse."""
import numpy as np
import pytest

from oracle import attn_oracle as A
from oracle import seq_oracle as O
from tests import attn_util as U
from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch
from tests.test_gpu_seq_outputs import Guarded, lens, same, scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def mods():
    from linear_rnn_sequence_wkv7_amd import groupnorm, layernorm, linattn
    return layernorm, linattn, groupnorm


H, EPS = 4, 64e-5


def layer_inputs(seed, B, T, Dk, Dv, dtype, shared=2):
    """v comes from the norm; q and k, which a layer projects from it too, are given."""
    rng = np.random.default_rng(seed)
    x = U.attn_inputs(seed, B, T, H, Dk, Dv, Hq=H // shared, Hk=H // shared, dtype=dtype, state=True)
    C = H * Dv
    r = lambda *s: rng.standard_normal(s)
    f = lambda a: a.astype(np.float32)
    x.update(x=S.as_dtype(r(B, T, C), dtype), res=S.as_dtype(r(B, T, C), dtype), gate=S.as_dtype(r(B, T, C), dtype), dy=S.as_dtype(r(B, T, C), dtype),
             dh=S.as_dtype(r(B, T, C), dtype), ds=f(r(B, H, Dk, Dv)), w1=f(1 + 0.2 * r(C)), b1=f(0.1 * r(C)), gw=f(1 + 0.2 * r(C)), gb=f(0.1 * r(C)),
             w2=f(1 + 0.2 * r(C)), b2=f(0.1 * r(C)))
    del x["v"]
    return x


def layer_forward(d, lengths=None):
    """Norm of the stream, attention, norm of the heads with its gate, and the next layer's norm."""
    ln, la, gn = mods()
    B, T, C = d["x"].shape
    n, h, m1, r1 = ln.layernorm_forward(d["x"], residual=d["res"], weight=d["w1"], bias=d["b1"], lengths=lengths)
    o, st = la.linattn_forward(d["q"], d["k"], n.view(B, T, H, C // H), d["g"], scale=0.25, state=d["state"], lengths=lengths)
    z, mg, rg = gn.groupnorm_forward(o.view(B * T, 1, C), H, weight=d["gw"], bias=d["gb"], gate=d["gate"].view(B * T, 1, C), act="silu", eps=EPS)
    y, h2, m2, r2 = ln.layernorm_forward(z.view(B, T, C), residual=h, weight=d["w2"], bias=d["b2"], lengths=lengths)
    return {"n": n, "h": h, "m1": m1, "r1": r1, "o": o, "state": st, "mg": mg, "rg": rg, "y": y, "h2": h2, "m2": m2, "r2": r2}


def layer_backward(d, f, lengths=None):
    ln, la, gn = mods()
    B, T, C = d["x"].shape
    flat = lambda t: t.view(B * T, 1, C)
    g2 = ln.layernorm_backward(f["h2"], d["dy"], f["m2"], f["r2"], weight=d["w2"], bias=d["b2"], dh=d["dh"], lengths=lengths)
    gg = gn.groupnorm_backward(flat(f["o"]), H, flat(g2["x"]), f["mg"], f["rg"], weight=d["gw"], bias=d["gb"], gate=flat(d["gate"]), act="silu")
    ga = la.linattn_backward(d["q"], d["k"], f["n"].view(B, T, H, C // H), d["g"], gg["x"].view(B, T, H, C // H), scale=0.25, state=d["state"],
                             dstate=d["ds"], lengths=lengths)
    g1 = ln.layernorm_backward(f["h"], ga["v"].view(B, T, C), f["m1"], f["r1"], weight=d["w1"], bias=d["b1"], dh=g2["h"], lengths=lengths)
    return {"x": g1["x"], "w1": g1["weight"], "b1": g1["bias"], "q": ga["q"], "k": ga["k"], "g": ga["g"], "state": ga["state"],
            "gate": gg["gate"].view(B, T, C), "gw": gg["weight"], "gb": gg["bias"], "w2": g2["weight"], "b2": g2["bias"]}


@pytest.mark.parametrize("B,T,Dk,Dv", [(2, 150, 16, 24), (1, 33, 20, 9), (1, 1, 8, 8)])
def test_training_chain(B, T, Dk, Dv):
    """Forward and every gradient in a row, fp32, against the chained oracle.  Each operator's result is
    within about 1e-5 of its terms' sizes (their own tests); the norms divide by a spread that these inputs
    keep above a hundredth of the values: 1e-3 of each result's largest value bounds the chain."""
    x = layer_inputs(T, B, T, Dk, Dv, "f32")
    d = {k: to_dev(v) for k, v in x.items()}
    f = layer_forward(d)
    g = layer_backward(d, f)
    torch().cuda.synchronize()
    C = H * Dv
    h = np.asarray(x["x"], np.float64) + x["res"]
    n, _, r1 = A.layer_forward(h, x["w1"], x["b1"])
    heads, flat = (lambda a: a.reshape(B, T, H, Dv)), (lambda a: np.asarray(a, np.float64).reshape(B * T, 1, C))
    o, st, _ = A.attn_forward(x["q"], x["k"], heads(n), x["g"], 0.25, x["state"])
    z, _, rg = O.norm_forward(flat(o), H, x["gw"], x["gb"], flat(x["gate"]), True, EPS)
    h2 = h + z.reshape(B, T, C)
    y, _, r2 = A.layer_forward(h2, x["w2"], x["b2"])
    for r, v in ((r1, h), (rg, o), (r2, h2)):
        assert np.max(r) * np.sqrt(np.mean(v ** 2)) < 100
    g2 = A.layer_backward(h2, x["dy"], x["w2"], x["dh"])
    gg = O.norm_backward(flat(o), H, flat(g2["h"]), x["gw"], x["gb"], flat(x["gate"]), True, EPS)
    ga = A.attn_backward(x["q"], x["k"], heads(n), x["g"], heads(gg["x"]), 0.25, x["state"], x["ds"])
    g1 = A.layer_backward(h, ga["v"].reshape(B, T, C), x["w1"], g2["h"])
    ref = {"x": g1["h"], "w1": g1["weight"], "b1": g1["bias"], "q": ga["q"], "k": ga["k"], "g": ga["g"], "state": ga["state"],
           "gate": gg["gate"].reshape(B, T, C), "gw": gg["weight"], "gb": gg["bias"], "w2": g2["weight"], "b2": g2["bias"]}
    for what, got, want in [("y", f["y"], y), ("stream", f["h2"], h2), ("state", f["state"], st)] + [("d" + k, g[k], ref[k]) for k in ref]:
        S.check(what, to_host(got), want, 1e-3 * np.max(np.abs(want)))


def token(d, state, stream, index):
    ln, la, gn = mods()
    B, C = d["x"].shape
    n, h, _, _ = ln.layernorm_forward(d["x"].view(B, 1, C), residual=stream.view(B, 1, C), weight=d["w1"], bias=d["b1"], h=stream.view(B, 1, C),
                                      return_stats=False)
    o = la.linattn_step(d["q"], d["k"], n.view(B, H, C // H), d["g"], state, scale=0.25, state_index=index)
    z, _, _ = gn.groupnorm_forward(o.view(B, 1, C), H, weight=d["gw"], bias=d["gb"], gate=d["gate"].view(B, 1, C), act="silu", eps=EPS, return_stats=False)
    y, _, _, _ = ln.layernorm_forward(z, residual=h, weight=d["w2"], bias=d["b2"], h=h, return_stats=False)
    return y


def test_serving_chain_in_a_graph():
    """Single tokens captured once and replayed with new inputs and other states each time, eager
    work and synchronisations between: every replay is the eager result."""
    t = torch()
    B, Dk, Dv, Sp = 6, 32, 16, 9
    x = layer_inputs(3, B, 1, Dk, Dv, "bf16")
    d = {k: to_dev(v[:, 0] if k in ("x", "q", "k", "g", "gate") else v) for k, v in x.items()}
    index = t.tensor([3, 0, -1, 8, 1, 5], dtype=t.int32, device="cuda")
    state0 = t.randn(Sp, H, Dk, Dv, device="cuda")
    stream0 = t.randn(B, H * Dv, device="cuda", dtype=t.bfloat16)
    state, stream = state0.clone(), stream0.clone()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        token(d, state.clone(), stream.clone(), index)
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y = token(d, state, stream, index)
    state.copy_(state0), stream.copy_(stream0)
    es, eh = state0.clone(), stream0.clone()
    for r in range(4):
        gen = t.Generator(device="cuda").manual_seed(r)
        for k in ("x", "q", "k"):
            d[k].copy_(t.randn(d[k].shape, generator=gen, device="cuda"))
        index.copy_(t.randperm(Sp, generator=gen, device="cuda")[:B])
        want = token(d, es, eh, index).clone()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(y, want) and t.equal(state, es) and t.equal(stream, eh), r


def test_prompt_then_tokens():
    """A layer over 70 tokens, and its prompt of 64 with six single tokens behind it, in fp32: the same y
    and state, up to a hundred units of the terms in attention and what the norms divide by (see above)."""
    t = torch()
    B, T, P, Dk, Dv = 2, 70, 64, 32, 16
    d = {k: to_dev(v) for k, v in layer_inputs(5, B, T, Dk, Dv, "f32").items()}
    whole = layer_forward(d)
    first = {k: (v[:, :P].contiguous() if k in ("x", "res", "q", "k", "g", "gate") else v) for k, v in d.items()}
    pool = layer_forward(first)["state"]
    ys = []
    for i in range(P, T):
        one = {k: (v[:, i].contiguous() if k in ("x", "q", "k", "g", "gate") else v) for k, v in d.items()}
        ys.append(token(one, pool, d["res"][:, i].contiguous(), None)[:, 0])
    t.cuda.synchronize()
    top = float(whole["y"].abs().max())
    assert float((t.stack(ys, 1) - whole["y"][:, P:]).abs().max()) <= 1e-3 * top
    assert float((pool - whole["state"]).abs().max()) <= 1e-5 * float(whole["state"].abs().max())


@pytest.mark.parametrize("T", [90, 700])
def test_training_chain_in_a_graph(T):
    """Forward and backward captured together, a ragged batch, replayed with other inputs."""
    t = torch()
    B, Dk, Dv = 3, 32, 16
    d = {k: to_dev(v) for k, v in layer_inputs(1, B, T, Dk, Dv, "bf16").items()}
    lengths = t.tensor([T, 0, 33], dtype=t.int32, device="cuda")

    def both():
        f = layer_forward(d, lengths)
        return f, layer_backward(d, f, lengths)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        both()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        f, g = both()
    for r in range(4):
        gen = t.Generator(device="cuda").manual_seed(r)
        for k in ("x", "res", "q", "k", "dy", "dh"):
            d[k].copy_(t.randn(d[k].shape, generator=gen, device="cuda"))
        lengths.copy_(t.tensor([[T, 0, 33], [1, T, 64], [0, 0, 0], [T - 1, 65, 16]][r], dtype=t.int32))
        ef, eg = both()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for k in ("y", "state", "o"):
            assert t.equal(f[k], ef[k]), (r, k)
        for k in g:
            assert t.equal(g[k], eg[k]), (r, k)


def test_two_graphs_share_a_workspace():
    """Two captured calls that use one workspace, replayed one after the other: each is its own result."""
    t = torch()
    la = mods()[1]
    B, T, Dk = 2, 600, 64
    ws = t.empty(max(la.linattn_workspace_bytes(B, T, H, Dk, Dk), la.linattn_backward_workspace_bytes(B, T, H, Dk, Dk)), dtype=t.uint8, device="cuda")
    ds = [{k: to_dev(v) for k, v in U.attn_inputs(s, B, T, H, Dk, Dk, dtype="bf16").items() if v is not None} for s in (1, 2)]
    args = lambda d: (d["q"], d["k"], d["v"], d["g"])
    run = lambda d: (la.linattn_forward(*args(d), workspace=ws), la.linattn_backward(*args(d), d["v"], workspace=ws))
    want = [run(d) for d in ds]
    t.cuda.synchronize()
    graphs, got = [], []
    for d in ds:
        graphs.append(t.cuda.CUDAGraph())
        with t.cuda.graph(graphs[-1]):
            got.append(run(d))
    for _ in range(3):
        for (y, st), g in got:
            for o in (y, st, *g.values()):
                o.zero_()
        for graph in graphs:
            graph.replay()
        t.cuda.synchronize()
        for ((y, st), g), ((ey, est), eg) in zip(got, want):
            same("y", y, ey), same("state", st, est)
            for k in g:
                same("d" + k, g[k], eg[k])


def test_two_streams_at_once():
    """The chain on two streams, each with its own inputs, equals itself alone."""
    t = torch()
    ds = [{k: to_dev(v) for k, v in layer_inputs(s, 2, 500, 64, 64, "bf16").items()} for s in (1, 2)]
    run = lambda d: (lambda f: (f["y"], layer_backward(d, f)))(layer_forward(d))
    alone = [run(d) for d in ds]
    t.cuda.synchronize()
    streams, out = [t.cuda.Stream(), t.cuda.Stream()], [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with t.cuda.stream(s):
                out[i].append(run(ds[i]))
    t.cuda.synchronize()
    for i in range(2):
        for y, g in out[i]:
            assert t.equal(y, alone[i][0])
            for k in g:
                assert t.equal(g[k], alone[i][1][k]), k


ATTN = [
    # B, T, H, Hq, Hk, Hv, Dk, Dv, dtype, lengths
    (2, 1, 3, 3, 3, 3, 5, 7, "f32", None),
    (2, 33, 4, 2, 1, 4, 24, 17, "bf16", [33, 0]),
    (3, 130, 2, 2, 2, 2, 64, 64, "bf16", [130, 1, 65]),
    (1, 700, 2, 1, 2, 1, 128, 64, "bf16", None),
    (2, 300, 2, 2, 1, 2, 100, 128, "f32", [299, 64]),
    (1, 2100, 2, 2, 2, 2, 128, 128, "bf16", [2077]),
    (1, 4200, 1, 1, 1, 1, 33, 64, "f32", None),
]


@pytest.mark.parametrize("case", ATTN, ids=["B{}_T{}_H{}_{}_{}_{}_D{}_{}_{}".format(*c[:9]) for c in ATTN])
def test_attention_between_guards(case):
    la = mods()[1]
    t = torch()
    B, T, H, Hq, Hk, Hv, Dk, Dv, dtype, lengths = case
    x = {k: to_dev(v) for k, v in U.attn_inputs(T, B, T, H, Dk, Dv, Hq, Hk, Hv, dtype=dtype, state=True).items()}
    dy, ds = t.randn(B, T, H, Dv, device="cuda").to(x["q"].dtype), t.randn(B, H, Dk, Dv, device="cuda")

    def calls(x, dy, ds, ln, o=None, ws=(None, None)):
        o = o or {}
        a, kw = (x["q"], x["k"], x["v"], x["g"]), dict(state=x["state"], lengths=ln, scale=0.3)
        y, s = la.linattn_forward(*a, **kw, y=o.get("y"), state_out=o.get("s"), workspace=ws[0])
        return y, s, la.linattn_backward(*a, dy, dstate=ds, **kw, grads=o.get("g"), workspace=ws[1])
    y, s, g = calls(x, dy, ds, lens(lengths))
    q = Guarded()
    heads = dict(Hq=Hq, Hk=Hk, Hv=Hv)
    ws, ws_ok = scratch(la.linattn_workspace_bytes(B, T, H, Dk, Dv, **heads))
    ws2, ws2_ok = scratch(la.linattn_backward_workspace_bytes(B, T, H, Dk, Dv, **heads))
    out = {"y": q.out(y), "s": q.out(s), "g": {k: q.out(v) for k, v in g.items()}}
    y2, s2, g2 = calls({k: q.put(v) for k, v in x.items()}, q.put(dy), q.put(ds), q.put(lens(lengths)), out, (ws, ws2))
    t.cuda.synchronize()
    same("y", y2, y)
    same("state", s2, s)
    for k in g:
        assert g2[k] is out["g"][k]
        same("d" + k, g2[k], g[k])
    q.check()
    assert ws_ok() and ws2_ok()
    state = x["state"].clone()   # in place
    la.linattn_forward(x["q"], x["k"], x["v"], x["g"], state=state, lengths=lens(lengths), scale=0.3, y=y2, state_out=state)
    same("y in place", y2, y), same("state in place", state, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lengths,Dk,Dv,state", [(512, [512, 511, 1], 20, 33, True), (513, [513, 512, 0], 40, 24, False), (1100, [1100, 1024, 1025], 24, 70, True),
                                                   (1024, None, 72, 20, True)])
@pytest.mark.parametrize("per_token", [True, False])
def test_gradients_of_decays_over_long_runs(T, lengths, Dk, Dv, state, per_token, dtype):
    """The gradient of g is summed in runs of 512 tokens: lengths at and beside their ends, with states and
    without, emptied ones among them.  The bound of one sum over all later tokens holds for the runs, too: a
    state's product with its gradient has no terms that the sum's magnitudes do not have."""
    la = mods()[1]
    t = torch()
    B, n = 3, 2
    x = U.attn_inputs(T, B, T, n, Dk, Dv, Hk=1, dtype=dtype, per_token=per_token, state=state, rate=0.1)
    if per_token:
        x["g"][:, 300, 0] = -np.inf
    rng = np.random.default_rng(T)
    dy, ds = S.as_dtype(rng.standard_normal((B, T, n, Dv)), dtype), rng.standard_normal((B, n, Dk, Dv)).astype(np.float32)
    g = la.linattn_backward(*(to_dev(x[k]) for k in "qkvg"), to_dev(dy), scale=0.3, state=None if not state else to_dev(x["state"]), dstate=to_dev(ds),
                            lengths=lens(lengths))
    t.cuda.synchronize()
    ref, tol = U.attn_grad_bounds(x, dy, ds, 0.3, lengths)
    for k in ("g", "state", "q", "k", "v"):
        S.check("d" + k, to_host(g[k]), ref[k], tol[k], bf16=g[k].dtype == t.bfloat16)


@pytest.mark.parametrize("B,T,H", [(0, 5, 2), (2, 0, 3), (2, 5, 0), (0, 0, 0)])
@pytest.mark.parametrize("constant", [False, True])
def test_attention_of_nothing(B, T, H, constant):
    """Without tokens the state and its gradient pass through, and constant decays have a gradient of 0."""
    la = mods()[1]
    t = torch()
    q, g = t.ones(B, T, H, 8, device="cuda"), t.zeros(*(() if constant else (B, T)), H, device="cuda")
    st, ds = t.randn(B, H, 8, 8, device="cuda"), t.randn(B, H, 8, 8, device="cuda")
    y, s = la.linattn_forward(q, q, q, g, state=st)
    gr = la.linattn_backward(q, q, q, g, q.clone(), state=st, dstate=ds)
    t.cuda.synchronize()
    assert y.shape == q.shape and all(gr[k].shape == q.shape for k in "qkv")
    assert t.equal(s, st) and t.equal(gr["state"], ds) and bool((gr["g"] == 0).all()) and gr["g"].shape == g.shape


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Dk,Dv", [(3, 2, 5, 7), (1, 4, 64, 64), (2, 3, 128, 100), (300, 4, 32, 64)])
def test_steps_between_guards(B, H, Dk, Dv, dtype):
    la = mods()[1]
    t = torch()
    x = {k: to_dev(v) for k, v in U.attn_inputs(B, B, 1, H, Dk, Dv, dtype=dtype, step=True).items() if v is not None}
    index, pool = t.randperm(B + 2, device="cuda")[:B].to(t.int32), t.randn(B + 2, H, Dk, Dv, device="cuda")
    a = pool.clone()
    y = la.linattn_step(x["q"], x["k"], x["v"], x["g"], a, state_index=index)
    q = Guarded()
    a2 = q.put(pool)
    y2 = la.linattn_step(*(q.put(x[k]) for k in "qkvg"), a2, state_index=q.put(index), y=q.out(y))
    none = la.linattn_step(*(q.put(x[k]) for k in "qkvg"), q.put(pool[:0]), state_index=q.put(index), y=q.out(y))
    t.cuda.synchronize()
    same("y", y2, y), same("pool", a2, a)
    assert bool((none == 0).all())
    q.check()


@pytest.mark.parametrize("x_dtype,h_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("B,T,C,lengths", [(3, 5, 7, None), (2, 40, 500, [40, 3]), (3, 33, 960, [0, 33, 1]), (2, 65, 2048, None), (1, 9, 4097, None), (2, 3, 9000, [3, 2]),
                                           (1, 4, 20000, None)])
def test_norm_between_guards(B, T, C, lengths, x_dtype, h_dtype):
    ln = mods()[0]
    t = torch()
    x = {k: to_dev(v) for k, v in U.norm_inputs(C, B, T, C, x_dtype, h_dtype).items()}
    dy, dh = t.randn(B, T, C, device="cuda").to(x["x"].dtype), t.randn(B, T, C, device="cuda").to(x["residual"].dtype)

    def calls(x, dy, dh, ls, o=None, ws=None):
        o = o or {}
        f = ln.layernorm_forward(x["x"], residual=x["residual"], weight=x["weight"], bias=x["bias"], lengths=ls, **{k: o.get(k) for k in ("y", "h", "mean", "rstd")})
        return f, ln.layernorm_backward(f[1], dy, f[2], f[3], weight=x["weight"], bias=x["bias"], dh=dh, lengths=ls, x_dtype=x_dtype, grads=o.get("g"), workspace=ws)
    f, g = calls(x, dy, dh, lens(lengths))
    q = Guarded()
    ws, ws_ok = scratch(ln.layernorm_backward_workspace_bytes(B, T, C))
    out = {n: q.out(v) for n, v in zip(("y", "h", "mean", "rstd"), f)}
    out["g"] = {k: q.out(v) for k, v in g.items() if k != "x" or x_dtype != h_dtype}
    f2, g2 = calls({k: q.put(v) for k, v in x.items()}, q.put(dy), q.put(dh), q.put(lens(lengths)), out, ws)
    t.cuda.synchronize()
    for n, a, b in zip(("y", "h", "mean", "rstd"), f2, f):
        same(n, a, b)
    for k in g:
        same("d" + k, g2[k], g[k])
    q.check()
    assert ws_ok()


def test_bindings_refuse():
    t = torch()
    ln, la, _ = mods()
    z = lambda *s, **k: t.zeros(*s, device="cuda", **k)
    q, g, st = z(2, 6, 4, 8), z(2, 6, 4), z(2, 4, 8, 8)
    one, g1 = z(2, 4, 8), z(2, 4)
    x, m = z(2, 6, 8), z(2, 6)
    cases = [
        (TypeError, lambda: la.linattn_forward(q.half(), q.half(), q.half(), g)),
        (TypeError, lambda: la.linattn_forward(q, q.bfloat16(), q, g)),
        (TypeError, lambda: la.linattn_forward(q, q, q, g.bfloat16())),
        (ValueError, lambda: la.linattn_forward(q, q[:, :5], q, g)),
        (ValueError, lambda: la.linattn_forward(q.transpose(1, 2), q, q, g)),
        (ValueError, lambda: la.linattn_forward(q, z(2, 6, 8, 8)[:, :, ::2], q, g)),
        (ValueError, lambda: la.linattn_forward(q, z(2, 6, 4, 7), q, g)),
        (ValueError, lambda: la.linattn_forward(z(2, 6, 3, 8), q, q, g)),
        (ValueError, lambda: la.linattn_forward(q, q, q, z(2, 5, 4))),
        (ValueError, lambda: la.linattn_forward(q, q, q, g, state=z(2, 4, 8, 7))),
        (TypeError, lambda: la.linattn_forward(q, q, q, g, state=st.bfloat16())),
        (ValueError, lambda: la.linattn_forward(q, q, q, g, lengths=z(3, dtype=t.int32))),
        (TypeError, lambda: la.linattn_forward(q, q, q, g, lengths=z(2, dtype=t.int64))),
        (ValueError, lambda: la.linattn_forward(q, q, q, g, y_dtype="f16")),
        (ValueError, lambda: la.linattn_forward(q, q, q, g, state=st.cpu())),
        (RuntimeError, lambda: la.linattn_forward(q, q, q, g, y=q)),
        (RuntimeError, lambda: la.linattn_forward(z(1, 2, 1, 129), z(1, 2, 1, 129), z(1, 2, 1, 8), z(1, 2, 1))),
        (RuntimeError, lambda: la.linattn_forward(q, q, q, g, scale=float("nan"))),
        (ValueError, lambda: la.linattn_step(one, one, one, g1, z(2, 4, 8, 7))),
        (ValueError, lambda: la.linattn_step(one, one, one, g1, st, state_index=z(3, dtype=t.int32))),
        (RuntimeError, lambda: la.linattn_step(one, one, one, g1, z(1, 4, 8, 8))),
        (ValueError, lambda: la.linattn_backward(q, q, q, g, z(2, 6, 4, 7))),
        (ValueError, lambda: la.linattn_backward(q, q, q, g, q.clone(), grads={"y": q})),
        (RuntimeError, lambda: la.linattn_backward(q, q, q, g, q.clone(), grads={"q": q})),
        (RuntimeError, lambda: la.linattn_backward(q, q, q, g, q.clone(), dstate=st, grads={"state": st})),
        (RuntimeError, lambda: la.linattn_backward(q, q, q, g, q.clone(), workspace=z(16, dtype=t.uint8))),
        (TypeError, lambda: ln.layernorm_forward(x.half())),
        (ValueError, lambda: ln.layernorm_forward(x, residual=z(2, 6, 7))),
        (ValueError, lambda: ln.layernorm_forward(x, h=x.clone())),
        (ValueError, lambda: ln.layernorm_forward(x, weight=z(7))),
        (TypeError, lambda: ln.layernorm_forward(x, weight=z(8, dtype=t.bfloat16))),
        (RuntimeError, lambda: ln.layernorm_forward(x, eps=0.0)),
        (RuntimeError, lambda: ln.layernorm_forward(x, residual=x.clone(), h=x)),
        (ValueError, lambda: ln.layernorm_forward(x[:, ::2])),
        (ValueError, lambda: ln.layernorm_backward(x, x.clone(), z(2, 5), m)),
        (TypeError, lambda: ln.layernorm_backward(x, x.clone(), m, m.clone(), dh=x.bfloat16())),
        (ValueError, lambda: ln.layernorm_backward(x, x.clone(), m, m.clone(), x_dtype="f16")),
        (RuntimeError, lambda: ln.layernorm_backward(x, x.clone(), m, m.clone(), grads={"h": x})),
        (RuntimeError, lambda: ln.layernorm_backward(x, x.clone(), m, m.clone(), weight=z(8), workspace=z(16, dtype=t.uint8))),
    ]
    for i, (err, fn) in enumerate(cases):
        with pytest.raises(err):
            fn()
            pytest.fail(f"case {i} was accepted")
