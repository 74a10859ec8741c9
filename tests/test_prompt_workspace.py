"""Workspace sizes of the prompt path, by the library's host-only queries."""
import ctypes

import pytest

from frame_level_delta_b200 import vda as V


def _decay_bytes(N, H, d, T, backward):
    w = H * d
    c, n = V.vda_decay_config(N, H, d, T, w, w, w, w, 1.0), ctypes.c_size_t(0)
    f = V.lib().vda_decay_attention_backward_workspace if backward else V.lib().vda_decay_attention_workspace
    assert f(ctypes.byref(c), ctypes.byref(n)) == V.VDA_OK
    return n.value


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("N,T", [(1024, 204800), (65535, 65535), (300, 1 << 20)])
def test_sequences_of_one_segment_take_no_workspace(N, T, backward):
    """A segment is at least 512 tokens, and only sequences of several leave states: two for
    each segment's tokens at most, however many sequences there are."""
    H, d = 24, 128
    per = H * d * d * 4 * (3 if backward else 1)
    n = _decay_bytes(N, H, d, T, backward)
    assert n % per == 0 and n <= 2 * (T // 512) * per
    # ... and a segment is a share of the work, about 148 of them in all, so with many heads few states.
    assert n <= 2 * 148 * H * d * d * 4


def test_long_sequences_keep_room_for_their_segments():
    """One sequence has as many segments as its tokens fill, the last in part."""
    H, d = 24, 128
    n = _decay_bytes(1, H, d, 11300, False) // (H * d * d * 4)
    assert 3 <= n <= 11300 // 512 + 1
    assert _decay_bytes(1, H, d, 1152, False) == 0
