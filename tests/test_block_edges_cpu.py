"""The decoder-block operators' host side at the ends of its ranges, without a GPU."""
import ctypes

import pytest
import torch

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


P = 0x20000  # a fake device address, never dereferenced
SHAPE = block_ops.Fp4Shape(16, 128)
CACHE = block_ops.Kv4Struct(2, 16, 2, 128, P, P, P, P)
CALLS = {  # arguments that launch nothing, and which of them have 32 bits
    "matvec": (block_ops._MATVEC, block_ops._matvec_args, [ctypes.addressof(SHAPE), P, P, P, 1, 128, 0, P, 0, 16, 0], [4, 6, 8]),
    "append": (block_ops._APPEND, block_ops._token_args, [ctypes.addressof(CACHE), P, P, 1, 256, 256, 0, P, 4, P, P, 0, 0, 0], [3, 6, 8, 11]),
    "gather": (block_ops._GATHER, block_ops._token_args, [ctypes.addressof(CACHE), P, P, 1, 256, 256, 0, P, 4, P, P, 0, 0, 0], [3, 6, 8, 11]),
    "attend": (block_ops._ATTEND, block_ops._attend_args,
               [ctypes.addressof(CACHE), P, 1, 512, 0, 4, P, 4, P, 1.0, 7, P, 512, P, P, 1 << 30, 0, 0], [2, 4, 5, 7, 10]),
    "norm": (block_ops._NORM, block_ops._norm_args, [0, 64, P, 1, 64, P, 0, 64, P, P, P, 0, 0, 1, 1.0, 1e-6, P, 64, P, 1, 64, 0],
             [0, 1, 3, 6, 11, 13, 19])}


@pytest.mark.parametrize("name,at", [(n, None) for n in CALLS] + [(n, at) for n, c in CALLS.items() for at in c[3]])
def test_a_word_past_32_bits_is_refused_and_not_cut(name, at):
    which, pack, args, _ = CALLS[name]
    if at is None:
        assert block_ops.lib().wd_call(which, pack(*args)) == 0
        return
    for past in (1 << 32, -(1 << 32), 1 << 62):  # what is left of it in 32 bits would be taken
        wide = list(args)
        wide[at] += past
        assert block_ops.lib().wd_call(which, pack(*wide)) == 2
        assert b"32 bits" in block_ops.lib().moe_last_error()


def test_tensors_whose_addresses_are_held_cannot_be_replaced():
    """Replaced tensors would leave the kernels on the old memory."""
    w = block_ops.Fp4Weights(16, 128, device="cpu")
    for name in ("codes", "scales"):
        with pytest.raises(AttributeError):
            setattr(w, name, torch.zeros_like(getattr(w, name)))
    assert w._ptrs == (w.codes.data_ptr(), w.scales.data_ptr())
    c = block_ops.Kv4Cache(2, 16, 1, 64, device="cpu")
    with pytest.raises(AttributeError):
        c.tensors = [t.clone() for t in c.tensors]
    with pytest.raises(TypeError):
        c.tensors[2] = c.tensors[2].clone()
    assert (c.struct.k_codes, c.struct.k_scales, c.struct.v_codes, c.struct.v_scales) == tuple(t.data_ptr() for t in c.tensors)


@pytest.mark.parametrize("N", [INT_MAX - 15, INT_MAX - 14, INT_MAX])
def test_the_most_rows(N):
    sh = ctypes.byref(block_ops.Fp4Shape(N, 32))
    assert block_ops.lib().wd_fp4_packed_bytes(sh, 0) == -(-N // 16) * 1024
    assert block_ops.lib().wd_fp4_packed_bytes(sh, 1) == -(-N // 16) * 64
