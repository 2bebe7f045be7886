"""Turned appends where results lie on borders between codes or next to them. The cache has to hold the nearest MXFP4 to the exact
turned key: codes and scales are compared for equality, against the product in 64 bits (off by 2^-52, far less than what the
magnitudes here put between a value and the border that it is next to)."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref
from .test_rope_gpu import _fill, _n, turned

pytestmark = pytest.mark.gpu


def _held(rope, case):
    cache, table, lens, cu, q, k, v, _ = case
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, torch.empty(q.shape, dtype=q.dtype, device="cuda"), cu)
    got = [torch.empty(k.shape, device="cuda") for _ in range(2)]
    block_ops.wd_kv4_gather(cache, table, lens, *got, cu)
    return [_n(t) for t in got]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("magnitude", [1 + 1e-9, 1 - 1e-9, -1 - 1e-9, 1 + 2.0 ** -40])
def test_magnitudes_that_are_one_in_fp32_only(magnitude, interleaved, kind):
    """What a turn by nothing leaves on a border, or on a power of two that decides the scale, the magnitude moves off it."""
    def edit(k, v):
        k[::3, 0, :32] = np.float32([4, 2.5, 0.25, 0.75, 1.25, 1.75, 3.5, -4]).repeat(4)
        k[1::3, 0, 32:64] = np.float32([7, 5, -5, -2.5, 3.5, 0.75, -1.75, -0.25]).repeat(4)
    case = _fill([300, 41], [0, 5], 2, 3, 128, 32, kind, seed=4, edit=edit)
    freqs = torch.zeros(32, dtype=torch.float64)
    got_k, got_v = _held(block_ops.Rope(freqs, interleaved, magnitude), case)
    k = _n(case[5])
    want = np.concatenate([k[..., :64] * magnitude, k[..., 64:]], -1)
    assert np.array_equal(got_k, ref.rounded(want)) and np.array_equal(got_v, ref.rounded(_n(case[6])))
    assert not np.array_equal(got_k, ref.rounded(k * np.sign(magnitude)))  # (the magnitude does decide some)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 16), (64, 48), (128, 80), (128, 16), (256, 112), (256, 240)])
def test_elements_that_do_not_turn_in_blocks_that_do(dim, rot, interleaved):
    """Half of a block turns: its scale may be a turned element's, and the other half's codes are of what was given, zeros and
    values on borders among them."""
    def edit(k, v):
        k[::2, 0, rot:] = 0
        k[1::2, 0, rot:] = np.float32([2.5, -0.25, 0.75, -5, 1.25, 0, 3.5, -1.75]).repeat(2)[np.arange(dim - rot) % 16]
        k[::3, 0, :rot] = np.float32([3, -1, 2, 0.5]).repeat(4)[np.arange(rot) % 16]
    case = _fill([500, 63], [0, 9], 2, 3, dim, 64, "bf16", seed=rot, edit=edit)
    freqs = block_ops.rope_freqs(rot)
    got_k, got_v = _held(block_ops.Rope(freqs, interleaved), case)
    want = turned(_n(case[5]), case[7], freqs.numpy(), interleaved)[0]
    assert np.array_equal(got_k, ref.rounded(want)) and np.array_equal(got_v, ref.rounded(_n(case[6])))
