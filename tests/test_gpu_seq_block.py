"""The scan, the convolution and the group norm as they are used together and with
the WKV recurrence: training and serving chains, captured into HIP graphs, on
other streams; and what their Python bindings refuse."""
import numpy as np
import pytest

from linear_rnn_sequence_wkv7_amd import inputs as G
from oracle import seq_oracle as O
from tests import seq_util as S
from tests.gpu_util import announce, dev_inputs, to_dev, to_host, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def mods():
    from linear_rnn_sequence_wkv7_amd import groupnorm, shortconv, ssm
    return shortconv, ssm, groupnorm


def block_inputs(seed, B, T, C, N, K, dtype):
    rng = np.random.default_rng(seed)
    x = S.scan_inputs(seed, B, T, C, N, 1, dtype)
    x.update(w=rng.standard_normal((C, K)).astype(np.float32) * 0.5, cb=rng.standard_normal(C).astype(np.float32) * 0.1,
             gw=(1 + 0.2 * rng.standard_normal(C)).astype(np.float32), gb=rng.standard_normal(C).astype(np.float32) * 0.1,
             gate=S.as_dtype(rng.standard_normal((B, T, C)), dtype), dy=S.as_dtype(rng.standard_normal((B, T, C)), dtype))
    return x


HEADS = 4


def block_forward(d, lengths=None, saved=None):
    """Convolution, scan, norm of the heads with its gate: what a layer does between its projections."""
    cv, sm, gn = mods()
    B, T, C = d["x"].shape
    u, cs = cv.shortconv_forward(d["x"], d["w"], bias=d["cb"], lengths=lengths)
    h, ss = sm.ssm_forward(u, d["dt"], d["A"], d["Bm"], d["Cm"], D=d["D"], dt_bias=d["dt_bias"], z=d["z"], lengths=lengths, checkpoints=saved)
    o, mean, rstd = gn.groupnorm_forward(h.view(B * T, 1, C), HEADS, weight=d["gw"], bias=d["gb"], gate=d["gate"].view(B * T, 1, C))
    return u, cs, h, ss, o.view(B, T, C), mean, rstd


def block_backward(d, fw, lengths=None, saved=None):
    cv, sm, gn = mods()
    B, T, C = d["x"].shape
    u, _, h, _, _, mean, rstd = fw
    flat = lambda t: t.view(B * T, 1, C)
    g = gn.groupnorm_backward(flat(h), HEADS, flat(d["dy"]), mean, rstd, weight=d["gw"], bias=d["gb"], gate=flat(d["gate"]))
    s = sm.ssm_backward(u, d["dt"], d["A"], d["Bm"], d["Cm"], g["x"].view(B, T, C), D=d["D"], dt_bias=d["dt_bias"], z=d["z"], lengths=lengths,
                        checkpoints=saved)
    c = cv.shortconv_backward(d["x"], d["w"], s["x"], bias=d["cb"], lengths=lengths)
    return {"x": c["x"], "w": c["w"], "cb": c["bias"], "dt": s["dt"], "A": s["A"], "B": s["B"], "C": s["C"], "D": s["D"],
            "dt_bias": s["dt_bias"], "z": s["z"], "gw": g["weight"], "gb": g["bias"], "gate": g["gate"].view(B, T, C)}


@pytest.mark.parametrize("B,T,C", [(2, 100, 64), (1, 17, 40)])
def test_training_chain(B, T, C):
    """Forward and every gradient of the three in a row, fp32, against the chained oracle.  Each
    operator's result is within about 1e-5 of its terms' sizes (their own tests); the norm divides by
    a head's spread, which these inputs keep above a hundredth of its values: 1e-3 of each result's
    largest value bounds the chain."""
    N = 16
    x = block_inputs(T, B, T, C, N, 4, "f32")
    d = {k: to_dev(v) for k, v in x.items()}
    saved = torch().empty(mods()[1].ssm_checkpoint_bytes(B, T, C, N), dtype=torch().uint8, device="cuda")
    fw = block_forward(d, saved=saved)
    g = block_backward(d, fw, saved=saved)
    torch().cuda.synchronize()
    u, cs, _ = O.conv_forward(x["x"], x["w"], x["cb"])
    kw = dict(D=x["D"], dt_bias=x["dt_bias"], z=x["z"])
    h, hs, _ = O.scan_forward(u, x["dt"], x["A"], x["Bm"], x["Cm"], **kw)
    flat = lambda a: np.asarray(a, np.float64).reshape(B * T, 1, C)
    o, _, rstd = O.norm_forward(flat(h), HEADS, x["gw"], x["gb"], flat(x["gate"]))
    assert np.max(rstd) * np.sqrt(np.mean(h ** 2)) < 100
    gn = O.norm_backward(flat(h), HEADS, flat(x["dy"]), x["gw"], x["gb"], flat(x["gate"]))
    gs = O.scan_backward(u, x["dt"], x["A"], x["Bm"], x["Cm"], gn["x"].reshape(B, T, C), **kw)
    gc = O.conv_backward(x["x"], x["w"], gs["x"], x["cb"])
    ref = {"x": gc["x"], "w": gc["w"], "cb": gc["bias"], "dt": gs["dt"], "A": gs["A"], "B": gs["B"], "C": gs["C"], "D": gs["D"],
           "dt_bias": gs["dt_bias"], "z": gs["z"], "gw": gn["weight"], "gb": gn["bias"], "gate": gn["gate"].reshape(B, T, C)}
    for what, got, want in [("y", fw[4], o.reshape(B, T, C)), ("conv state", fw[1], cs), ("scan state", fw[3], hs)] + \
                           [("d" + k, g[k], ref[k]) for k in ref]:
        S.check(what, to_host(got), want, 1e-3 * np.max(np.abs(want)))


def test_norm_of_the_wkv_heads():
    """The recurrence's output, normalised per head and gated, against the oracle on that output."""
    from linear_rnn_sequence_wkv7_amd import groupnorm, wkv7
    wl = G.workload("fwd_bf16_b8_t1024_h32_d64", B=2, T=70, H=4, H_kv=4)
    d = dev_inputs(G.make_inputs(wl))
    y, _ = wkv7.wkv7_forward(d["r"], d["w"], d["k"], d["v"], d["a"], d["b"], y_dtype="f32")
    B, T, H, D = y.shape
    rng = np.random.default_rng(0)
    gate, w, b = (rng.standard_normal(s).astype(np.float32) for s in ((B * T, 1, H * D), (H * D,), (H * D,)))
    o, mean, rstd = groupnorm.groupnorm_forward(y.view(B * T, 1, H * D), H, weight=to_dev(w), bias=to_dev(b), gate=to_dev(gate), eps=64e-5)
    torch().cuda.synchronize()
    (ref, m_ref, r_ref), (tol, m_tol, r_tol) = S.norm_bounds(to_host(y).reshape(B * T, 1, H * D), H, w, b, gate, False, 64e-5, None)
    S.check("o", to_host(o), ref, tol)
    S.check("mean", to_host(mean), m_ref, m_tol)


def serving(d, cstate, sstate, index):
    cv, sm, gn = mods()
    u = cv.shortconv_step(d["x"], d["w"], cstate, bias=d["cb"], state_index=index)
    h = sm.ssm_step(u, d["dt"], d["A"], d["Bm"], d["Cm"], sstate, D=d["D"], dt_bias=d["dt_bias"], z=d["z"], state_index=index)
    o, _, _ = gn.groupnorm_forward(h[:, None], HEADS, weight=d["gw"], bias=d["gb"], gate=d["gate"][:, None], return_stats=False)
    return o


def step_inputs(B, C, N, K, Sp):
    x = block_inputs(B, B, 1, C, N, K, "bf16")
    d = {k: to_dev(v[:, 0] if k in ("x", "dt", "Bm", "Cm", "z", "gate") else v) for k, v in x.items() if k != "dy"}
    rng = np.random.default_rng(1)
    return d, to_dev(S.as_dtype(rng.standard_normal((Sp, K - 1, C)), "bf16")), to_dev(rng.standard_normal((Sp, C, N)).astype(np.float32))


def test_serving_chain_in_a_graph():
    """Single tokens captured once and replayed with new inputs and other states each time, eager
    work and synchronisations between: every replay is the eager result."""
    t = torch()
    B, C, N, K, Sp = 6, 64, 16, 4, 9
    d, cs, ss = step_inputs(B, C, N, K, Sp)
    index = t.tensor([3, 0, -1, 8, 1, 5], dtype=t.int32, device="cuda")
    cs0, ss0 = cs.clone(), ss.clone()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        serving(d, cs.clone(), ss.clone(), index)
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        o = serving(d, cs, ss, index)
    cs.copy_(cs0), ss.copy_(ss0)
    ecs, ess = cs0.clone(), ss0.clone()
    for r in range(4):
        gen = t.Generator(device="cuda").manual_seed(r)
        d["x"].copy_(t.randn(B, C, generator=gen, device="cuda"))
        index.copy_(t.randperm(Sp, generator=gen, device="cuda")[:B])
        want = serving(d, ecs, ess, index).clone()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(o, want) and t.equal(cs, ecs) and t.equal(ss, ess), r


def test_training_chain_in_a_graph():
    """Forward and backward captured together, a ragged batch, replayed with other inputs."""
    t = torch()
    B, T, C, N = 3, 90, 64, 16
    d = {k: to_dev(v) for k, v in block_inputs(1, B, T, C, N, 4, "bf16").items()}
    lengths = t.tensor([90, 0, 33], dtype=t.int32, device="cuda")
    saved = t.empty(mods()[1].ssm_checkpoint_bytes(B, T, C, N), dtype=t.uint8, device="cuda")

    def both():
        fw = block_forward(d, lengths, saved)
        return fw, block_backward(d, fw, lengths, saved)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        both()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        fw, g = both()
    for r in range(4):
        gen = t.Generator(device="cuda").manual_seed(r)
        for k in ("x", "dt", "z", "Bm", "Cm", "dy"):
            d[k].copy_(t.randn(d[k].shape, generator=gen, device="cuda"))
        lengths.copy_(t.tensor([[90, 0, 33], [1, 90, 64], [0, 0, 0], [89, 65, 16]][r], dtype=t.int32))
        efw, eg = both()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(fw[4], efw[4]) and t.equal(fw[1], efw[1]) and t.equal(fw[3], efw[3]), r
        for k in g:
            assert t.equal(g[k], eg[k]), (r, k)


def test_two_streams_at_once():
    """The chain on two streams, each with its own inputs, equals itself alone."""
    t = torch()
    B, T, C, N = 2, 200, 64, 16
    ds = [{k: to_dev(v) for k, v in block_inputs(s, B, T, C, N, 4, "bf16").items()} for s in (1, 2)]
    alone = []
    for d in ds:
        fw = block_forward(d)
        alone.append((fw[4], block_backward(d, fw)))
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    out = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with t.cuda.stream(s):
                fw = block_forward(ds[i])
                out[i].append((fw[4], block_backward(ds[i], fw)))
    t.cuda.synchronize()
    for i in range(2):
        for y, g in out[i]:
            assert t.equal(y, alone[i][0])
            for k in g:
                assert t.equal(g[k], alone[i][1][k]), k


def test_bindings_by_torchs_public_names(monkeypatch):
    """The public names of the current stream and device give what the short ways give, on a side stream too."""
    t = torch()
    from linear_rnn_sequence_wkv7_amd import _marshal
    cv, _, _ = mods()
    d = {k: to_dev(v) for k, v in block_inputs(1, 2, 40, 64, 16, 4, "bf16").items()}
    want, _ = cv.shortconv_forward(d["x"], d["w"], bias=d["cb"])
    side = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        assert _marshal._public_stream(side.device_index) == side.cuda_stream == _marshal._raw_stream(side.device_index)
    monkeypatch.setattr(_marshal, "_raw_stream", _marshal._public_stream)
    monkeypatch.setattr(_marshal, "_device", t.cuda.current_device)
    with t.cuda.stream(side):
        got, _ = cv.shortconv_forward(d["x"], d["w"], bias=d["cb"])
    t.cuda.synchronize()
    assert t.equal(got, want)


def test_bindings_refuse():
    t = torch()
    cv, sm, gn = mods()
    z = lambda *s, **k: t.zeros(*s, device="cuda", **k)
    x, A, Bm, w = z(2, 6, 8), z(8, 4), z(2, 6, 1, 4), z(8, 4)
    half = z(2, 6, 8, dtype=t.float16)
    cases = [
        (TypeError, lambda: sm.ssm_forward(half, half, A, Bm.half(), Bm.half())),
        (TypeError, lambda: sm.ssm_forward(x, x.bfloat16(), A, Bm, Bm)),
        (ValueError, lambda: sm.ssm_forward(x, x[:, :5], A, Bm, Bm)),
        (ValueError, lambda: sm.ssm_forward(x.transpose(0, 1), x, A, Bm, Bm)),
        (ValueError, lambda: sm.ssm_forward(x, z(2, 12, 8)[:, ::2], A, Bm, Bm)),
        (ValueError, lambda: sm.ssm_forward(x, x, z(7, 4), Bm, Bm)),
        (TypeError, lambda: sm.ssm_forward(x, x, A.double(), Bm, Bm)),
        (ValueError, lambda: sm.ssm_forward(x, x, A, z(2, 6, 3, 4), z(2, 6, 3, 4))),
        (ValueError, lambda: sm.ssm_forward(x, x, A, Bm, Bm, lengths=z(3, dtype=t.int32))),
        (TypeError, lambda: sm.ssm_forward(x, x, A, Bm, Bm, lengths=z(2, dtype=t.int64))),
        (ValueError, lambda: sm.ssm_forward(x, x, A, Bm, Bm, y_dtype="f16")),
        (ValueError, lambda: sm.ssm_forward(x, x, A, Bm, Bm, checkpoints=z(10, dtype=t.uint8))),
        (ValueError, lambda: sm.ssm_forward(x, x, A, Bm, Bm, state=t.zeros(2, 8, 4))),
        (RuntimeError, lambda: sm.ssm_forward(x, x, A, Bm, Bm, y=x)),
        (RuntimeError, lambda: sm.ssm_forward(x, x, z(8, 65), z(2, 6, 1, 65), z(2, 6, 1, 65))),
        (ValueError, lambda: sm.ssm_step(x[:, 0].contiguous(), x[:, 0].contiguous(), A, Bm[:, 0].contiguous(), Bm[:, 0].contiguous(), z(2, 8, 5))),
        (RuntimeError, lambda: sm.ssm_step(x[:, 0].contiguous(), x[:, 0].contiguous(), A, Bm[:, 0].contiguous(), Bm[:, 0].contiguous(), z(1, 8, 4))),
        (RuntimeError, lambda: sm.ssm_backward(x, x, A, Bm, Bm, x, workspace=z(16, dtype=t.uint8))),
        (ValueError, lambda: cv.shortconv_forward(x, w, act="gelu")),
        (RuntimeError, lambda: cv.shortconv_forward(x, z(8, 5))),
        (TypeError, lambda: cv.shortconv_forward(x, w, state=z(2, 3, 8, dtype=t.bfloat16))),
        (ValueError, lambda: cv.shortconv_step(x[:, 0].contiguous(), w, z(2, 2, 8))),
        (ValueError, lambda: gn.groupnorm_forward(x, 3)),
        (ValueError, lambda: gn.groupnorm_forward(x, 2, gate=z(2, 6, 4))),
        (RuntimeError, lambda: gn.groupnorm_forward(x, 2, eps=0.0)),
        (ValueError, lambda: gn.groupnorm_backward(x, 2, x, z(2, 3), z(2, 2))),
    ]
    for i, (err, fn) in enumerate(cases):
        with pytest.raises(err):
            fn()
            pytest.fail(f"case {i} was accepted")
