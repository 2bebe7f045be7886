"""Block norms at the ends of their arguments' ranges."""
import pytest
import torch

from output_centric_expert_gb300 import block_ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 4864])
def test_the_most_tokens(T):
    """The last row and a step over all resident rows pass 2^31 (one channel: 4 GB each way)."""
    res = torch.arange(1, 252, device="cuda").to(torch.uint8).repeat(T // 251 + 1)[:T].to(torch.bfloat16)[:, None]
    out = torch.zeros_like(res)
    block_ops.wd_block_norm(res, out)
    assert torch.equal(res, out)
