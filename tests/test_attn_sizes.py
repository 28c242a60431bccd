"""Size queries and limits of linear attention that follow from what a call launches (CPU only)."""
import os
import subprocess
import sys

import pytest

from linear_rnn_sequence_wkv7_amd import linattn as L
from linear_rnn_sequence_wkv7_amd import wkv7 as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(not os.path.exists(W.lib_path()), reason="libwkv7.so not built")


@pytest.mark.parametrize("B,T,H,Dk,Dv", [(256, 1, 64, 128, 128), (4096, 16, 16, 8, 8), (64, 512, 32, 64, 64), (64, 512, 32, 128, 64)])
def test_short_sequences_keep_no_states(B, T, H, Dk, Dv):
    """Up to 512 tokens the gradients' workspace holds numbers for tokens and heads, and no state for either."""
    assert L.linattn_backward_workspace_bytes(B, T, H, Dk, Dv) <= B * H * (8 * T + 32) + 4096


def test_longer_ones_keep_two_for_every_further_512_tokens():
    at = lambda T: L.linattn_backward_workspace_bytes(64, T, 32, 64, 64)
    states = 64 * 32 * 2 * 64 * 64 * 4
    for n in range(1, 5):
        assert n * states <= at(512 * n + 1) <= at(512 * (n + 1)) <= n * states + 64 * 32 * (8 * 512 * (n + 1) + 32 * (n + 2)) + 4096


# B, T, H, Hq, Hk, Hv, Dk, Dv; whether a call runs
MANY = [
    ((32, 16384, 64, 64, 64, 64, 128, 128), True),    # 2^32 elements of each array, nothing shared
    ((32, 16384, 64, 64, 64, 64, 127, 128), True),
    ((32, 16384, 64, 16, 16, 64, 128, 128), True),    # sums of 2^30 elements in fours
    ((64, 16384, 64, 32, 64, 64, 128, 128), True),    # 2^32 in fours: 2^30 threads
    ((128, 16384, 64, 64, 32, 64, 126, 128), False),  # as many one by one
    ((1 << 24, 1, 1, 1, 1, 1, 1, 1), False),          # 3 x 512 threads for each sequence
    ((2, 1 << 29, 16, 16, 16, 16, 1, 1), False),      # a thread for each of 2^34 decays
]
CHILD = """
import ctypes
from linear_rnn_sequence_wkv7_amd import linattn as L
from linear_rnn_sequence_wkv7_amd import wkv7 as W
lib = L._lib()
for n in {cases!r}:
    B, T, H, Hq, Hk, Hv, Dk, Dv = n
    d = L.LinattnDesc(B, T, H, Hq, Hk, Hv, Dk, Dv, 1, 1, 1, 0, 1.0, 0, None)
    need = lib.linattn_backward_workspace_bytes(ctypes.byref(d))
    at = iter(range(1 << 45, 1 << 50, 1 << 45))   # far apart, and never read: there is no device
    p = lambda: ctypes.c_void_p(next(at))
    rc = lib.linattn_backward(ctypes.byref(d), p(), p(), p(), p(), None, p(), None, p(), p(), p(), p(), None, p(), need, None)
    print(rc, W.load_library().wkv7_last_error().decode().replace(chr(10), " "))
"""


def test_gradients_are_refused_by_the_launches_they_need():
    """A call of less than 2^32 threads in each of its launches passes every check in front of the one for a
    device, of which the child sees none; no sums are counted where no heads share an operand."""
    env = {**os.environ, "HIP_VISIBLE_DEVICES": "-1", "ROCR_VISIBLE_DEVICES": "-1"}
    r = subprocess.run([sys.executable, "-c", CHILD.format(cases=[n for n, _ in MANY])], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.splitlines()
    assert len(lines) == len(MANY)
    for (n, runs), line in zip(MANY, lines):
        code, message = line.split(" ", 1)
        if runs:
            assert int(code) == W.WKV7_EDEVICE, (n, line)
        else:
            assert int(code) == W.WKV7_EUNSUPPORTED and "2^32" in message, (n, line)
