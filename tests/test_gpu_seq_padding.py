"""Padding behind a sequence's end, where what the sequence itself brings is not finite:
its y and its gradients are 0 all the same."""
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


def mods():
    from linear_rnn_sequence_wkv7_amd import groupnorm, shortconv, ssm
    return shortconv, ssm, groupnorm


def lens(lengths):
    return torch().tensor(lengths, dtype=torch().int32, device="cuda")


def padding_is_zero(what, t, lengths):
    got = to_host(t)
    for b, n in enumerate(lengths):
        assert np.all(got[b, n:] == 0), f"{what}: padding of sequence {b}"


SCANS = [(16, 16, 1), (40, 16, 1), (40, 16, 200), (300, 16, 1), (40, 32, 1), (40, 64, 1), (90, 8, 300), (40, 15, 1)]   # T, N, copies


def scan_case(T, N, copies, z, bad):
    """Four sequences, `copies` times, two of them from states with one value that is not finite."""
    C = 24
    x = S.scan_inputs(T + N, 4, T, C, N, 1, "f32", z=z, state=True)
    x["state"][0, 3, 1] = x["state"][1, 3, 0] = bad
    rep = lambda v: None if v is None else to_dev(np.concatenate([v] * copies))
    a = (rep(x["x"]), rep(x["dt"]), to_dev(x["A"]), rep(x["Bm"]), rep(x["Cm"]))
    lengths = [T - 3, 5, 0, T - 9] * copies
    return a, dict(D=to_dev(x["D"]), dt_bias=to_dev(x["dt_bias"]), z=rep(x["z"]), state=rep(x["state"]), lengths=lens(lengths)), lengths, rep, C


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("z", [True, False])
@pytest.mark.parametrize("T,N,copies", SCANS)
def test_scan_forward(T, N, copies, z, bad):
    """For each number of waves to a block of channels."""
    a, kw, lengths, _, _ = scan_case(T, N, copies, z, bad)
    y, s = mods()[1].ssm_forward(*a, **kw)
    torch().cuda.synchronize()
    padding_is_zero("y", y, lengths)
    s = to_host(s)
    assert not np.isfinite(s[0, 3, 1])
    assert np.all(np.isfinite(s[2])) and np.all(np.isfinite(s[:, 4:]))   # an empty sequence, other channels


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("z", [True, False])
@pytest.mark.parametrize("T,N,copies", SCANS)
def test_scan_backward(T, N, copies, z, bad):
    """For each number of runs; gradients of the state that are not finite too."""
    a, kw, lengths, rep, C = scan_case(T, N, copies, z, bad)
    rng = np.random.default_rng(T)
    dy, ds = rng.standard_normal((4, T, C)).astype(np.float32), rng.standard_normal((4, C, N)).astype(np.float32)
    ds[0, 5, 0] = ds[3, 5, 1] = bad
    g = mods()[1].ssm_backward(*a, rep(dy), dstate=rep(ds), **kw)
    torch().cuda.synchronize()
    for k in ("x", "dt", "z", "B", "C"):
        if g[k] is not None:
            padding_is_zero("d" + k, g[k], lengths)
    assert np.all(np.isfinite(to_host(g["state"])[:, 0])) and np.all(np.isfinite(to_host(g["dt_bias"])[[0, 1, 2, 4]]))


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_convolution(dtype, bad):
    cv, _, _ = mods()
    B, T, C, K = 3, 37, 24, 4
    rng = np.random.default_rng(1)
    x, dy = (S.as_dtype(rng.standard_normal((B, T, C)), dtype) for _ in range(2))
    w, bias = rng.standard_normal((C, K)).astype(np.float32), rng.standard_normal(C).astype(np.float32)
    w[2, 1] = w[5, 3] = bias[7] = bad
    lengths = [20, 0, 36]
    kw = dict(bias=to_dev(bias), lengths=lens(lengths))
    y, _ = cv.shortconv_forward(to_dev(x), to_dev(w), **kw)
    g = cv.shortconv_backward(to_dev(x), to_dev(w), to_dev(dy), **kw)
    torch().cuda.synchronize()
    padding_is_zero("y", y, lengths)
    padding_is_zero("dx", g["x"], lengths)


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("T,C,G", [(1, 64, 2), (1, 30, 2), (9, 24, 3), (9, 22, 1), (3000, 96, 2), (1, 4096, 1)])
def test_norm(T, C, G, bad):
    _, _, gn = mods()
    B = 3
    rng = np.random.default_rng(C)
    x, dy, gate = (rng.standard_normal((B, T, C)).astype(np.float32) for _ in range(3))
    weight, bias = rng.standard_normal(C).astype(np.float32), rng.standard_normal(C).astype(np.float32)
    weight[1], bias[C - 1] = bad, bad
    lengths = [T // 2, 0, T]
    kw = dict(weight=to_dev(weight), bias=to_dev(bias), gate=to_dev(gate), act="silu", lengths=lens(lengths))
    y, mean, rstd = gn.groupnorm_forward(to_dev(x), G, **kw)
    g = gn.groupnorm_backward(to_dev(x), G, to_dev(dy), mean, rstd, **kw)
    torch().cuda.synchronize()
    padding_is_zero("y", y, lengths)
    padding_is_zero("dx", g["x"], lengths)
    padding_is_zero("dgate", g["gate"], lengths)
