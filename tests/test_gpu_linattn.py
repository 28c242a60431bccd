"""Linear attention with a decay for each head on the GPU against the fp64 oracle: prompts, gradients and
steps over head sizes, lengths, shared heads, types, decays and padding."""
import numpy as np
import pytest

from oracle import attn_oracle as O
from tests import attn_util as A
from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch

pytestmark = pytest.mark.gpu
EPS32 = 2.0 ** -16   # of a whole fp32 result's norm: far above sums of whole operands, far below a bf16 operand's 2^-9


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def mod():
    from linear_rnn_sequence_wkv7_amd import linattn
    return linattn


def dev(x):
    return {k: to_dev(v) for k, v in x.items()}


def near(what, got, ref):
    """An fp32 result as a whole."""
    assert np.linalg.norm(to_host(got) - ref) <= EPS32 * np.linalg.norm(ref) + 1e-30, what


def forward(x, scale=0.5, lengths=None, y_dtype=None, whole=True, **kw):
    """Run, compare, and return what the library gave."""
    d = dev(x)
    y, st = mod().linattn_forward(d["q"], d["k"], d["v"], d["g"], scale=scale, state=d["state"], lengths=to_dev(lengths), y_dtype=y_dtype, **kw)
    torch().cuda.synchronize()
    (y_ref, s_ref), (y_tol, s_tol) = A.attn_bounds(x, scale, lengths)
    S.check("y", to_host(y), y_ref, y_tol, bf16=y.dtype == torch().bfloat16)
    S.check("state", to_host(st), s_ref, s_tol)
    if whole:
        near("state", st, s_ref)
    return y, st


def backward(x, dy, dstate=None, scale=0.5, lengths=None, **kw):
    d = dev(x)
    g = mod().linattn_backward(d["q"], d["k"], d["v"], d["g"], to_dev(dy), scale=scale, state=d["state"], dstate=to_dev(dstate),
                               lengths=to_dev(lengths), **kw)
    torch().cuda.synchronize()
    ref, tol = A.attn_grad_bounds(x, dy, dstate, scale, lengths)
    for n in ref:
        S.check("d" + n, to_host(g[n]), ref[n], tol[n], bf16=g[n].dtype == torch().bfloat16)
    near("dstate", g["state"], ref["state"])
    return g


def grads_of(x, dtype, seed=9, dstate=True):
    rng = np.random.default_rng(seed)
    B, T, H = x["q"].shape[0], x["q"].shape[1], x["g"].shape[-1]
    Dk, Dv = x["q"].shape[3], x["v"].shape[3]
    return S.as_dtype(rng.standard_normal((B, T, H, Dv)), dtype), rng.standard_normal((B, H, Dk, Dv)).astype(np.float32) if dstate else None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0, 1, 2, 15, 17, 31, 32, 33, 63, 64, 65, 96, 127, 129, 200])
def test_lengths(T, dtype):
    forward(A.attn_inputs(T, 2, T, 2, 64, 64, dtype=dtype, state=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (3, 5), (8, 8), (16, 4), (37, 61), (48, 80), (60, 64), (64, 65), (66, 64), (99, 128), (128, 1), (127, 127), (128, 128)])
def test_head_sizes(Dk, Dv, dtype):
    x = A.attn_inputs(Dk, 2, 70, 3, Dk, Dv, dtype=dtype, state=True)
    forward(x)
    backward(x, *grads_of(x, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0, 1, 2, 31, 33, 63, 64, 65, 129, 200])
def test_gradients(T, dtype):
    x = A.attn_inputs(T, 2, T, 2, 64, 128, dtype=dtype, state=True)
    g = backward(x, *grads_of(x, dtype))
    if T == 0:
        assert g["q"].numel() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hk,Hv", [(1, 1, 4), (2, 2, 4), (4, 1, 1), (1, 2, 4), (4, 4, 2)])
def test_shared_heads(Hq, Hk, Hv, dtype):
    x = A.attn_inputs(Hq, 2, 75, 4, 24, 40, Hq, Hk, Hv, dtype=dtype, state=True)
    forward(x)
    backward(x, *grads_of(x, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_constant_decays(dtype):
    """One decay a head: its gradient is the sum over the batch and the tokens."""
    x = A.attn_inputs(0, 3, 150, 5, 32, 32, dtype=dtype, per_token=False, state=True)
    forward(x, lengths=np.array([150, 0, 70], np.int32))
    backward(x, *grads_of(x, dtype), lengths=np.array([150, 0, 70], np.int32))
    backward(x, *grads_of(x, dtype, dstate=False))


@pytest.mark.parametrize("lengths", [[100, 0, 37, -5], [64, 65, 1, 1000], [0, 0, 0, 0]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding(lengths, dtype):
    """Whatever padding holds."""
    x = A.attn_inputs(1, 4, 100, 3, 40, 64, dtype=dtype, state=True)
    dy, ds = grads_of(x, dtype)
    lengths = np.array(lengths, np.int32)
    bad = {k: v.copy() if v is not None else None for k, v in x.items()}
    dy_bad = dy.copy()
    for b, n in enumerate(lengths):
        n = min(max(n, 0), 100)
        for a in (bad["q"], bad["k"], bad["v"], dy_bad):
            a[b, n:] = 0x7FC0 if dtype == "bf16" else np.nan
        bad["g"][b, n:] = np.inf
    clean = lambda a: a
    y, st = forward(x, lengths=lengths)
    d = dev(bad)
    y2, st2 = mod().linattn_forward(d["q"], d["k"], d["v"], d["g"], scale=0.5, state=d["state"], lengths=to_dev(lengths))
    assert torch().equal(y, y2) and torch().equal(st, st2)
    g = backward(x, dy, ds, lengths=lengths)
    g2 = mod().linattn_backward(d["q"], d["k"], d["v"], d["g"], to_dev(dy_bad), scale=0.5, state=d["state"], dstate=to_dev(ds), lengths=to_dev(lengths))
    for n in g:
        assert torch().equal(g[n], g2[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_of_every_size(dtype):
    """No decay at all, total ones (also several to a chunk, and at its ends), steep ones, growth."""
    x = A.attn_inputs(3, 2, 200, 4, 32, 32, dtype=dtype, state=True, rate=1.0)
    g = x["g"]
    g[:, :, 0] = 0.0
    g[:, [0, 5, 6, 31, 32, 63, 64, 100, 150, 199], 1] = -np.inf
    g[:, :, 2] *= 40
    g[:, 10:20, 2] = -1e30
    g[:, :, 3] = np.abs(g[:, :, 3]) * 0.01
    forward(x)
    backward(x, *grads_of(x, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_of_decays_lose_nothing(dtype):
    """A steep token early in a chunk leaves the later tokens' decays as they were: a running sum of -3000 in
    32 bits would move them by 1e-4."""
    x = A.attn_inputs(4, 1, 64, 1, 64, 64, dtype=dtype, rate=0.02)
    x["g"][:, 3] = -1300.0
    x["g"][:, 7] = -1300.0
    d = dev(x)
    y, st = mod().linattn_forward(d["q"], d["k"], d["v"], d["g"], y_dtype="f32")
    ref, s_ref, _ = O.attn_forward(x["q"], x["k"], x["v"], x["g"])
    near("y", y, ref)
    near("state", st, s_ref)


@pytest.mark.parametrize("y_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (33, 20)])
def test_types(Dk, Dv, dtype, y_dtype):
    """y and dy of the other type."""
    x = A.attn_inputs(5, 2, 90, 4, Dk, Dv, 4, 2, 4, dtype=dtype, state=True)
    y, _ = forward(x, y_dtype=y_dtype)
    assert y.dtype == (torch().float32 if y_dtype == "f32" else torch().bfloat16)
    backward(x, *grads_of(x, y_dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,T", [(1, 1, 1000), (3, 2, 700), (1, 8, 4200)])
def test_parts_side_by_side(B, H, T, dtype):
    """Few heads: sequences in many segments, of which some are padding."""
    x = A.attn_inputs(T, B, T, H, 24, 16, dtype=dtype, state=True, rate=0.02)
    lengths = None if B == 1 else np.array([T, 130, 0], np.int32)
    forward(x, lengths=lengths)
    backward(x, *grads_of(x, dtype), lengths=lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_heads_in_one_part(dtype):
    x = A.attn_inputs(6, 40, 70, 16, 8, 12, dtype=dtype, state=True)
    forward(x)
    backward(x, *grads_of(x, dtype))


def test_long_sequence_keeps_its_accuracy():
    """16384 tokens, memories of 10 to 1000 of them: y, the state, and the gradient of g (a sum over all
    later tokens) as whole results."""
    rng = np.random.default_rng(0)
    B, T, H, D = 1, 16384, 2, 32
    x = A.attn_inputs(7, B, T, H, D, D, dtype="bf16", rate=0.0)
    x["g"] = -(np.array([0.1, 0.001]) * np.exp(0.3 * rng.standard_normal((B, T, H)))).astype(np.float32)
    dy, ds = grads_of(x, "bf16")
    d = dev(x)
    _, st = mod().linattn_forward(d["q"], d["k"], d["v"], d["g"])
    g = mod().linattn_backward(d["q"], d["k"], d["v"], d["g"], to_dev(dy), dstate=to_dev(ds))
    _, s_ref, _ = O.attn_forward(x["q"], x["k"], x["v"], x["g"])
    ref = O.attn_backward(x["q"], x["k"], x["v"], x["g"], dy, dstate=ds)
    near("state", st, s_ref)
    near("dstate", g["state"], ref["state"])
    near("dg", g["g"], ref["g"])


def test_outputs_given_and_in_place():
    t = torch()
    x = A.attn_inputs(8, 2, 100, 3, 32, 48, dtype="bf16", state=True)
    d = dev(x)
    y, st = forward(x)
    y2, state = t.full_like(y, float("nan")), d["state"].clone()
    ws = t.full((mod().linattn_workspace_bytes(2, 100, 3, 32, 48),), 255, dtype=t.uint8, device="cuda")
    y3, st3 = mod().linattn_forward(d["q"], d["k"], d["v"], d["g"], scale=0.5, state=state, y=y2, state_out=state, workspace=ws)
    assert y3 is y2 and st3 is state and t.equal(y2, y) and t.equal(state, st)
    _, none = mod().linattn_forward(d["q"], d["k"], d["v"], d["g"], scale=0.5, state=d["state"], return_state=False)
    assert none is None
    dy, ds = grads_of(x, "bf16")
    g = backward(x, dy, ds)
    given = {n: t.full_like(v, float("nan")) for n, v in g.items()}
    ws = t.full((mod().linattn_backward_workspace_bytes(2, 100, 3, 32, 48),), 255, dtype=t.uint8, device="cuda")
    g2 = mod().linattn_backward(d["q"], d["k"], d["v"], d["g"], to_dev(dy), scale=0.5, state=d["state"], dstate=to_dev(ds), grads=given, workspace=ws)
    for n in g:
        assert g2[n] is given[n] and t.equal(g2[n], g[n]), n
    g3 = mod().linattn_backward(d["q"], d["k"], d["v"], d["g"], to_dev(dy), scale=0.5, state=d["state"], dstate=to_dev(ds), return_dg=False, return_dstate=False)
    assert g3["g"] is None and g3["state"] is None and t.equal(g3["k"], g["k"])


def test_gradients_against_differences():
    """Central differences of the library's own forward, in fp32: for a step e along a direction of length 1
    in every input, the loss (a sum of n terms of size s) is off by about U s sqrt(n), the quotient by that over e, and the
    third order by e^2 times the third derivative: below 1e-2 of the slope here for e = 1e-2."""
    t = torch()
    x = A.attn_inputs(11, 1, 70, 2, 16, 16, state=True)
    d = dev(x)
    dy, ds = grads_of(x, "f32")
    g = mod().linattn_backward(d["q"], d["k"], d["v"], d["g"], to_dev(dy), state=d["state"], dstate=to_dev(ds))

    def loss(m):
        y, st = mod().linattn_forward(m["q"], m["k"], m["v"], m["g"], state=m["state"])
        return float((y.double() * to_dev(dy).double()).sum() + (st.double() * to_dev(ds).double()).sum())
    for n in ("q", "k", "v", "g", "state"):
        way = g[n] / g[n].norm()   # the steepest direction
        e = 1e-2
        up, down = loss({**d, n: d[n] + e * way}), loss({**d, n: d[n] - e * way})
        slope = (up - down) / (2 * e)
        assert abs(slope - float(g[n].norm())) <= 1e-2 * float(g[n].norm()), n


# ---------------------------------------------------------------- steps

def step(x, pool, index=None, scale=0.5, y_dtype=None):
    d = dev({**x, "state": pool})
    y = mod().linattn_step(d["q"], d["k"], d["v"], d["g"], d["state"], scale=scale, state_index=to_dev(index), y_dtype=y_dtype)
    torch().cuda.synchronize()
    ref, after = O.attn_step(x["q"], x["k"], x["v"], x["g"], pool, index, scale)
    m, ma = O.attn_step(x["q"], x["k"], x["v"], x["g"], pool, index, scale, mag=True)
    # a decay: an exponential, 4 U; a sum of Dk products
    S.check("y", to_host(y), ref, (x["q"].shape[2] + 20) * S.U * m, bf16=y.dtype == torch().bfloat16)
    S.check("pool", to_host(d["state"]), after, 8 * S.U * ma)
    untouched = np.all(after == pool, axis=(1, 2, 3))
    assert np.array_equal(to_host(d["state"])[untouched], pool[untouched].astype(np.float64))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Dk,Dv", [(1, 1, 1, 1), (1, 32, 64, 64), (3, 4, 37, 61), (40, 16, 64, 64), (40, 16, 128, 128), (70, 9, 100, 127), (600, 1, 8, 5)])
def test_step(B, H, Dk, Dv, dtype):
    x = A.attn_inputs(B, B, 1, H, Dk, Dv, dtype=dtype, step=True)
    rng = np.random.default_rng(B)
    pool = rng.standard_normal((B + 3, H, Dk, Dv)).astype(np.float32)
    step(x, pool)
    index = rng.permutation(B + 3)[:B].astype(np.int32)
    step(x, pool, index)
    index[B // 2:] = rng.integers(-2, B + 5, B - B // 2)   # missing, out of range, the same twice
    step(x, pool, index, y_dtype="f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_shares_heads_and_constant_decays(dtype):
    x = A.attn_inputs(2, 6, 1, 4, 48, 32, 1, 2, 4, dtype=dtype, step=True, per_token=False)
    x["g"][1] = -np.inf
    step(x, np.random.default_rng(0).standard_normal((6, 4, 48, 32)).astype(np.float32), np.array([5, 4, 3, 3, 3, 0], np.int32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_are_the_forward(dtype):
    """Twenty steps on a pool and one call over twenty tokens, both within their bounds of the oracle."""
    T, B, H = 20, 3, 2
    x = A.attn_inputs(12, B, T, H, 40, 24, dtype=dtype, state=True)
    (y_ref, s_ref), (y_tol, s_tol) = A.attn_bounds(x, 0.5)
    d = dev(x)
    pool = d["state"].clone()
    ys = [mod().linattn_step(*(d[n][:, t].contiguous() for n in "qkvg"), pool, scale=0.5) for t in range(T)]
    S.check("y", to_host(torch().stack(ys, 1)), y_ref, y_tol, bf16=dtype == "bf16")
    S.check("state", to_host(pool), s_ref, s_tol)
    forward(x)
