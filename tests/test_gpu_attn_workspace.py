"""Workspaces of linear attention at their smallest: between guards, where none is needed and where some is."""
import pytest

from tests.gpu_util import announce, torch
from tests.test_gpu_seq_outputs import scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def inputs(B, T, H, Dk, Dv, dtype, constant):
    t = torch()
    dt = t.float32 if dtype == "f32" else t.bfloat16
    r = lambda *s: t.randn(*s, device="cuda")
    return (r(B, T, H, Dk).to(dt), r(B, T, H, Dk).to(dt), r(B, T, H, Dv).to(dt), -r(*(() if constant else (B, T)), H).abs()), r(B, T, H, Dv).to(dt), \
        r(B, H, Dk, Dv), r(B, H, Dk, Dv)


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [0, 16, 256])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (128, 64), (128, 128)])
def test_without_tokens_no_workspace_is_written(Dk, Dv, size, dtype, constant):
    """None is needed, so one of any size may be given: every state's gradient passes through and the bytes stay."""
    from linear_rnn_sequence_wkv7_amd import linattn as la
    t = torch()
    B, H = 3, 5
    args, dy, st, ds = inputs(B, 0, H, Dk, Dv, dtype, constant)
    assert la.linattn_backward_workspace_bytes(B, 0, H, Dk, Dv) == 0
    whole = t.full((1 << 20,), 255, dtype=t.uint8, device="cuda")   # more than any write that starts within it could reach
    ws = whole[1 << 19:(1 << 19) + size]
    for state, dstate in ((st, ds), (None, ds), (st, None)):
        g = la.linattn_backward(*args, dy, state=state, dstate=dstate, workspace=ws)
        t.cuda.synchronize()
        assert bool((whole == 255).all())
        assert t.equal(g["state"], ds if dstate is not None else t.zeros_like(ds)) and bool((g["g"] == 0).all())
    y, s = la.linattn_forward(*args, state=st, workspace=ws)
    t.cuda.synchronize()
    assert bool((whole == 255).all()) and t.equal(s, st)


def test_gradients_of_more_than_2_32_elements():
    """The state is emptied 150 tokens before the end, so that the oracle needs no more than those."""
    from linear_rnn_sequence_wkv7_amd import linattn as la
    from tests import attn_util as A
    from tests.test_gpu_attn_large import decays
    from tests.test_gpu_seq_large import check, host, normal
    t = torch()
    T, H, D, N = 1050000, 64, 64, 150
    q, k, v, dy, g = *(normal(i, 1, T, H, D) for i in range(4)), decays(4, 1, T, H)
    assert q.numel() > 1 << 32
    g[:, T - N] = -1e5
    ds = normal(6, 1, H, D, D, dtype="f32")
    gr = la.linattn_backward(q, k, v, g, dy, scale=0.2, dstate=ds)
    t.cuda.synchronize()
    hs, last = slice(H - 2, H), slice(T - N, T)
    part = lambda x: x[:, last, hs]
    x = {**{n: host(part(a)) for n, a in (("q", q), ("k", k), ("v", v), ("g", g))}, "state": None}
    ref, tol = A.attn_grad_bounds(x, host(part(dy)), host(ds[:, hs]), 0.2)
    for n in ("q", "k", "v", "g"):
        check("d" + n, part(gr[n]), ref[n], tol[n])
    del q, k, v, dy, g, gr
    t.cuda.empty_cache()
