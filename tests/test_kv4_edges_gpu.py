"""The 4-bit KV cache at the ends of its arguments' ranges."""
import pytest
import torch

from .test_kv4_gpu import Filled, _attend, _q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 64, 2 ** 31 - 1])
@pytest.mark.parametrize("lens", [[5], [300, 0, 77], [9000, 40]])
def test_a_window_past_every_key_is_no_window(lens, window):
    f = Filled(lens, 2, 128, 16)
    q = _q(f.rng, len(lens), 16, 128)
    for a, b in zip(_attend(f, q, window=window), _attend(f, q)):
        assert torch.equal(a, b)
