"""GPU parity of the scan, the convolution and the group norm where y or dy has the
other type than x: fp32 inputs with bf16 y and dy, bf16 inputs with fp32 y and dy."""
import numpy as np
import pytest

from tests import seq_util as S
from tests.gpu_util import announce, to_dev, to_host, torch

pytestmark = pytest.mark.gpu

OTHER = {"f32": "bf16", "bf16": "f32"}


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
    return (d["x"], d["dt"], d["A"], d["Bm"], d["Cm"]), dict(D=d["D"], dt_bias=d["dt_bias"], z=d["z"], state=d["state"])


def lens(lengths):
    return None if lengths is None else torch().tensor(lengths, dtype=torch().int32, device="cuda")


SCANS = [
    # B, T, C, N, G, lengths: one, four and eight waves to a block of channels; odd and even rows and groups
    (3, 15, 37, 16, 1, None),
    (2, 50, 21, 20, 3, [50, 11]),
    (2, 40, 6, 64, 6, None),
    (3, 50, 37, 16, 1, [33, 0, 50]),
    (2, 64, 35, 12, 5, None),
    (2, 60, 30, 3, 2, None),
    (2, 130, 37, 16, 1, [130, 71]),
    (3, 200, 45, 8, 5, None),
    (2, 140, 32, 16, 2, [99, 140]),
    (2, 300, 18, 16, 18, None),
]
SCAN_IDS = ["B{}_T{}_C{}_N{}_G{}".format(*c[:5]) for c in SCANS]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SCANS, ids=SCAN_IDS)
def test_scan_forward(case, dtype):
    """A bf16 y behind fp32 inputs whose rows are odd starts on 2 bytes only."""
    B, T, C, N, G, lengths = case
    x = S.scan_inputs(T * 5 + C, B, T, C, N, G, dtype, state=True)
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(x, T, lengths, True, B=B, Cg=C // G)
    a, kw = dev_args(x)
    y, s = M().ssm_forward(*a, **kw, lengths=lens(lengths), y_dtype=OTHER[dtype])
    torch().cuda.synchronize()
    assert y.dtype == (torch().bfloat16 if dtype == "f32" else torch().float32)
    S.check("y", to_host(y), y_ref, y_tol, bf16=dtype == "f32")
    S.check("state", to_host(s), s_ref, s_tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,N,G", [(37, 16, 1), (21, 5, 3), (64, 16, 2)])
def test_scan_step(C, N, G, dtype):
    B = 5
    x = S.scan_inputs(C, B, 1, C, N, G, dtype, step=True)
    pool = np.random.default_rng(C).standard_normal((B, C, N)).astype(np.float32)
    a, kw = dev_args(x)
    kw["state"] = st = to_dev(pool)
    y = M().ssm_step(*a, y_dtype=OTHER[dtype], **kw)
    torch().cuda.synchronize()
    one = {k: v[:, None] if k in ("x", "dt", "Bm", "Cm", "z") else v for k, v in x.items()}
    one["state"] = pool
    (y_ref, s_ref), (y_tol, s_tol) = S.scan_bounds(one, 1, None, True)
    S.check("y", to_host(y), y_ref[:, 0], y_tol[:, 0], bf16=dtype == "f32")
    S.check("state", to_host(st), s_ref, s_tol)
