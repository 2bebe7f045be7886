"""Ends of the ranges of rotary positions, the append with rotation and the attention of chunks that are refused before a launch."""
import ctypes

import pytest

from output_centric_expert_gb300 import block_ops

from .test_new_tokens_cpu import APPEND, CHUNK, P, SHAPE, UNSUPPORTED, _rotation


@pytest.mark.parametrize("magnitude", [1e-50, -1e-40, 2.0 ** -101, 5e-324])
def test_magnitudes_that_fp32_does_not_hold(magnitude):
    """FP32 has them with fewer bits or as 0: a key times one would not be the exact turned key, however large it is."""
    a = dict(r=_rotation(magnitude=magnitude), x=P, type=1, ldx=256, T=2, heads=4, dim=64, pos=P, out=P + 4096, ldo=256)
    assert block_ops.lib().wd_rope(*a.values(), None) == UNSUPPORTED
    a = APPEND | dict(r=_rotation(magnitude=magnitude))
    c = ctypes.byref(block_ops.Kv4Struct(*a.pop("sizes"), *[a.pop("arrays")] * 4))
    assert block_ops.lib().wd_kv4_rope_append(c, *a.values(), None) == UNSUPPORTED


MOST = 2 ** 31 - 2 ** 16  # of tokens, and of sequences: the first that a call refuses


@pytest.mark.parametrize("T,S", [(MOST, 2), (2 ** 31 - 1, 2), (3, MOST), (3, 2 ** 31 - 1)])
def test_tokens_and_sequences_next_to_2_31(T, S):
    """The tokens of a run behind the last one, and the sequences of a step behind the last, have to fit 32 bits."""
    a = APPEND | dict(T=T, S=S)
    sizes, arrays = (2, 16, 1, 64), a.pop("arrays")
    del a["sizes"]
    c = ctypes.byref(block_ops.Kv4Struct(*sizes, *[arrays] * 4))
    assert block_ops.lib().wd_kv4_rope_append(c, *a.values(), None) == SHAPE
    for fn in ("wd_kv4_append", "wd_kv4_gather"):
        assert getattr(block_ops.lib(), fn)(c, P, P, 1, 64, 64, T, P, 4, P, P, S, None, None) == SHAPE
    a = CHUNK | dict(T=T, S=S, q_heads=1)
    assert block_ops.lib().wd_kv4_attend_chunk(c, *a.values(), None) == SHAPE
