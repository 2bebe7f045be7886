"""Ends of the ranges of rotary positions, the append with rotation and the attention of chunks that are refused before a launch."""
import ctypes

import pytest

from output_centric_expert_gb300 import block_ops

from .test_new_tokens_cpu import APPEND, P, UNSUPPORTED, _rotation


@pytest.mark.parametrize("magnitude", [1e-50, -1e-40, 2.0 ** -101, 5e-324])
def test_magnitudes_that_fp32_does_not_hold(magnitude):
    """FP32 has them with fewer bits or as 0: a key times one would not be the exact turned key, however large it is."""
    a = dict(r=_rotation(magnitude=magnitude), x=P, type=1, ldx=256, T=2, heads=4, dim=64, pos=P, out=P + 4096, ldo=256)
    assert block_ops.lib().wd_rope(*a.values(), None) == UNSUPPORTED
    a = APPEND | dict(r=_rotation(magnitude=magnitude))
    c = ctypes.byref(block_ops.Kv4Struct(*a.pop("sizes"), *[a.pop("arrays")] * 4))
    assert block_ops.lib().wd_kv4_rope_append(c, *a.values(), None) == UNSUPPORTED
