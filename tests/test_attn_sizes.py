"""Size queries and limits of linear attention that follow from what a call launches (CPU only)."""
import os

import pytest

from linear_rnn_sequence_wkv7_amd import linattn as L
from linear_rnn_sequence_wkv7_amd import wkv7 as W

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
