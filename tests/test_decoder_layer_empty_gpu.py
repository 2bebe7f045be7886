"""A decoder layer whose batch has no rows, as a scheduler's iteration may have: nothing to do, and no error."""
import pytest
import torch

from .test_decoder_layer_extend_gpu import layer  # noqa: F401
from .test_decoder_layer_gpu import layer as plain_layer  # noqa: F401

pytestmark = pytest.mark.gpu


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[], [3, 0]])
def test_extend_without_rows(layer, lens, dtype):  # noqa: F811
    """No sequences at all, and sequences without new tokens."""
    held, err = [t.clone() for t in layer.cache.tensors], _ints(0)
    res = torch.zeros(0, layer.w.moe.shape.H, dtype=dtype, device="cuda")
    table = torch.zeros(len(lens), 2, dtype=torch.int32, device="cuda")
    out = layer.extend(res, table, _ints(*lens), _ints(*[0] * (len(lens) + 1)), err)
    assert out is res and int(err) == 0 and all(torch.equal(a, b) for a, b in zip(held, layer.cache.tensors))


@pytest.mark.parametrize("rope", [False, True])
def test_step_without_rows(layer, plain_layer, rope):  # noqa: F811
    made, err = layer if rope else plain_layer, _ints(0)
    res = torch.zeros(0, made.w.moe.shape.H, dtype=torch.bfloat16, device="cuda")
    assert made.step(res, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), _ints(), err) is res and int(err) == 0
