"""What linear attention holds of a value that is no bf16: inputs whose results are exact in
fp32, so that y has to be them to the bit, and their one rounding where y is bf16."""
import numpy as np
import pytest

from tests.gpu_util import announce, torch

pytestmark = pytest.mark.gpu
SIZES = [(64, 64), (128, 128), (64, 128), (128, 64), (37, 61), (100, 24)]
TIE = 1 + 2.0 ** -8               # halfway between two bf16
NEAR_TIES = {TIE + 2.0 ** -18: 1 + 2.0 ** -7, 1 + 3 * 2.0 ** -8 - 2.0 ** -18: 1 + 2.0 ** -7}   # value: the bf16 next to it


@pytest.fixture(autouse=True)
def _gpu_and_name(request):
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    announce(request.node.nodeid)
    yield


def forward(dtype, Dk, Dv, T, y_dtype, scale=1.0, state=None, keys=True):
    """One head, no decay; q is column t % Dk's unit vector (with keys: the first's, as are k's), v column t % Dv's."""
    from linear_rnn_sequence_wkv7_amd import linattn
    t = torch()
    at, rows = t.arange(T, device="cuda"), t.zeros(1, T, 1, Dk, device="cuda")
    q, k, v = rows.clone(), rows.clone(), t.zeros(1, T, 1, Dv, device="cuda")
    q[0, at, 0, at * 0 if keys else at % Dk] = 1
    k[0, at, 0, 0] = 1 if keys else 0
    v[0, at, 0, at % Dv] = 1
    dt = t.float32 if dtype == "f32" else t.bfloat16
    y, _ = linattn.linattn_forward(q.to(dt), k.to(dt), v.to(dt), t.zeros(1, device="cuda"), scale=scale, state=state, y_dtype=y_dtype)
    return y[0, :, 0].double()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", SIZES)
def test_y_has_all_bits_of_the_state(Dk, Dv, dtype):
    """k is 0, so that y is a row of the state in front of the first token."""
    t, T = torch(), 150
    state = t.randn(1, 1, Dk, Dv, device="cuda", generator=t.Generator("cuda").manual_seed(Dk))
    want = state[0, 0].double()[t.arange(T, device="cuda") % Dk]
    assert t.equal(forward(dtype, Dk, Dv, T, "f32", state=state, keys=False), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", SIZES)
def test_y_has_all_bits_of_products_within_a_chunk(Dk, Dv, dtype):
    """Every product of a query and a key is 1 and P the scale, a number of 24 bits: y is the scale in the columns that v had."""
    t, T, scale = torch(), min(Dv, 32), float(np.float32(0.7371912))
    want = t.zeros(T, Dv, device="cuda", dtype=t.float64)
    for i in range(T):
        want[i, :i + 1] = scale
    assert t.equal(forward(dtype, Dk, Dv, T, "f32", scale=scale), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", NEAR_TIES)
@pytest.mark.parametrize("Dk,Dv", SIZES)
def test_y_is_rounded_once(Dk, Dv, value, dtype):
    """Values beside the middle of two bf16 go to the nearer one: of the state, and of P."""
    t = torch()
    state = t.full((1, 1, Dk, Dv), value, device="cuda")
    assert bool((state.double() == value).all())
    assert bool((forward(dtype, Dk, Dv, 70, "bf16", state=state, keys=False) == NEAR_TIES[value]).all())
    y = forward(dtype, Dk, Dv, min(Dv, 32), "bf16", scale=value)
    assert set(y.unique().tolist()) <= {0.0, NEAR_TIES[value]} and float(y[0, 0]) == NEAR_TIES[value]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("g", [-0.01, -0.5, -2.0, -5.0, -10.0, -20.0])
def test_gradient_of_decays_is_off_by_its_terms_rounding(g, D, dtype):
    """Whatever the decay leaves of the difference: a term's sum of about 30 accumulations is off by the root of that many
    roundings, and the terms are added from either end of up to 512 tokens, 11 times one's error in the middle of a
    random walk that is held at both: 6 * 11 * sqrt(2) units, less than 2^-17 of <q, dq>, as norms."""
    from linear_rnn_sequence_wkv7_amd import linattn
    from oracle import attn_oracle as O
    from oracle.seq_oracle import as_f64
    from tests import attn_util as A
    from tests import seq_util as S
    from tests.gpu_util import to_dev, to_host
    x = A.attn_inputs(1, 1, 512, 2, D, D, dtype=dtype, rate=0.0)
    x["g"][:] = np.float32(g)
    dy = S.as_dtype(np.random.default_rng(2).standard_normal((1, 512, 2, D)), dtype)
    got = linattn.linattn_backward(*(to_dev(x[n]) for n in "qkvg"), to_dev(dy), scale=D ** -0.5)["g"]
    ref = O.attn_backward(x["q"], x["k"], x["v"], x["g"], dy, D ** -0.5)
    terms = (as_f64(x["q"]) * ref["q"]).sum(-1)
    assert np.linalg.norm(to_host(got) - ref["g"]) <= 2.0 ** -17 * np.linalg.norm(terms)
