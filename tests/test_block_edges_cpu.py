"""The decoder-block operators' host side at the ends of its ranges, without a GPU."""
import ctypes

import pytest

from output_centric_expert_gb300 import block_ops

INT_MAX = 2 ** 31 - 1


def _ctas(S, q_heads, max_blocks, window, sizes=(4096, 16, 8, 128)):
    return block_ops.lib().wd_kv4_attend_ctas(ctypes.byref(block_ops.Kv4Struct(*sizes)), S, q_heads, max_blocks, window)


@pytest.mark.parametrize("window", [INT_MAX - 64, INT_MAX - 63, INT_MAX - 62, INT_MAX - 1, INT_MAX])
@pytest.mark.parametrize("S,q_heads", [(1, 8), (1, 128), (3, 32), (64, 64), (64, 128), (700, 8)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_window_past_every_key_launches_what_no_window_does(S, q_heads, dim, window):
    sizes = (4096, 16, 8, dim)
    most = _ctas(1000, 64, 1000, 0, sizes)  # 2 CTAs per SM, what the workspace is sized for
    for blocks in (1, 2, 9, 512):
        n = _ctas(S, q_heads, blocks, window, sizes)
        assert 0 < n <= most and n == _ctas(S, q_heads, blocks, 0, sizes)


def test_attend_launches_no_more_ctas_than_tiles():
    assert _ctas(1, 8, 1, 0) == 8  # 16 keys of 8 heads: a tile each
    assert _ctas(0, 8, 1, 0) == 0
    assert _ctas(1, 8, 1000, 1) == 8 and _ctas(1, 8, 1000, 300) == 16  # 256 keys a tile
    for bad in ((-1, 8, 1, 0), (1, 7, 1, 0), (1, 8, 0, 0), (1, 8, 1, -1)):
        assert _ctas(*bad) == 0


@pytest.mark.parametrize("S,q_heads,blocks,window", [
    (INT_MAX, 8, INT_MAX, 0), (INT_MAX, INT_MAX // 8 * 8, INT_MAX, INT_MAX), (1 << 20, 8 << 10, 1 << 20, 0), (1 << 20, 8, 1 << 20, 0)])
def test_more_tiles_than_are_counted_are_refused(S, q_heads, blocks, window):
    """Products of the sizes that pass 32 and 64 bits."""
    assert _ctas(S, q_heads, blocks, window) == 0


def test_attend_refuses_more_tiles_than_it_counts():
    P = 0x20000  # a fake device address, never dereferenced
    c = ctypes.byref(block_ops.Kv4Struct(2, 16, 8, 128, P, P, P, P))
    assert block_ops.lib().wd_kv4_attend(c, P, 1, 1024, 1 << 20, 8, P, 1 << 20, P, 1.0, 0, P, 1024, P, P, 1 << 40, None, None) == 2
    assert b"capacity" in block_ops.lib().moe_last_error()
