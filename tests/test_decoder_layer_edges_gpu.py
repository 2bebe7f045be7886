"""Decode steps with slots that hold no sequence and lengths that have no place."""
import pytest
import torch

from .test_decoder_layer_gpu import layer  # noqa: F401

pytestmark = pytest.mark.gpu


def _step(layer, lens, table, seed=0):
    torch.manual_seed(seed)
    for t in layer.cache.tensors:
        t.zero_()
    res = torch.randn(len(lens), layer.w.moe.shape.H, device="cuda").to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.step(res, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), err)
    return res, int(err)


@pytest.mark.parametrize("length,row", [(64, [5, 6]), (10 ** 6, [5, 6]), (2 ** 31 - 1, [5, 6]), (-1, [5, 6]), (-100, [5, 6]), (0, [-1, -1]), (17, [5, -1])])
def test_a_slot_out_of_range_is_flagged_and_disturbs_nobody(layer, length, row):  # noqa: F811
    """Past the rotations' tables, negative, or an idle slot without pages: the other sequences' results stay."""
    table = torch.tensor([[0, 1], row, [2, 3]], dtype=torch.int32, device="cuda")
    res, err = _step(layer, [3, length, 20], table)
    assert err == 1 and torch.isfinite(res.float()).all()
    table[1] = torch.tensor([5, 6])
    want, err = _step(layer, [3, 9, 20], table)
    assert err == 0
    assert torch.equal(res[0], want[0]) and torch.equal(res[2], want[2])


def test_lengths_past_the_rotations_but_inside_the_cache(layer):  # noqa: F811
    """max_positions is 64, the row holds 80 tokens."""
    table = torch.tensor([[0, 1, 2, 3, 4]], dtype=torch.int32, device="cuda")
    assert _step(layer, [63], table)[1] == 0
    assert _step(layer, [64], table)[1] == 1
