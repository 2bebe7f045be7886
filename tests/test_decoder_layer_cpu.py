"""What a decode step does with lengths before any kernel sees them, on CPU tensors."""
import pytest
import torch

from output_centric_expert_gb300.decoder_layer import DecoderLayer


@pytest.mark.parametrize("lens,rows,flag", [
    ([0, 7], [0, 7], 0), ([8], [7], 1), ([3, -1], [3, 0], 1), ([2 ** 31 - 1, -2 ** 31, 5], [7, 0, 5], 1)])
def test_lengths_outside_the_rotations_are_flagged_and_index_nothing(lens, rows, flag):
    layer = object.__new__(DecoderLayer)
    angle = torch.arange(8.0)[:, None] * torch.ones(4)
    layer.cos, layer.sin = angle.cos(), angle.sin()
    err = torch.zeros(1, dtype=torch.int32)
    pos = layer._positions(torch.tensor(lens, dtype=torch.int32), err)
    assert pos.tolist() == rows and err.tolist() == [flag]
    assert layer._positions(torch.tensor(lens, dtype=torch.int32), None).tolist() == rows
    err.fill_(2)  # other bits stay
    layer._positions(torch.tensor(lens, dtype=torch.int32), err)
    assert err.tolist() == [2 | flag]
    x = torch.randn(len(lens), 3, 8)
    want = torch.cat([torch.cat((x[i:i + 1, :, :4] * angle[r].cos() - x[i:i + 1, :, 4:] * angle[r].sin(),
                                 x[i:i + 1, :, 4:] * angle[r].cos() + x[i:i + 1, :, :4] * angle[r].sin()), -1) for i, r in enumerate(rows)])
    layer._rotate(x, pos)
    assert torch.allclose(x, want)
