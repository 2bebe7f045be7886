"""Bits and range of the attention of several new tokens: what its logits, probabilities and keys have to hold at the ends of what
its description allows. Tolerances as in test_chunk_gpu, but for what a test says itself."""
import numpy as np
import pytest
import torch

from .test_chunk_gpu import Chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group,new", [(64, 2, 30), (128, 4, 90), (256, 1, 40)])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_no_scale_with_large_keys(scale, dim, group, new):
    """Logits of 0 whatever the keys, up to 2^100: every key weighs the same."""
    def edit(k, v):
        k[:] = 2.0 ** 99
        k[::2] *= -1
        v[::2] = np.abs(v[::2])
    c = Chunk([70], [new], 2, group, dim, 16, edit=edit)
    c.q.fill_(1.0)
    c.check(*c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dim,new", [(64, 40), (128, 40), (128, 300), (256, 40)])
def test_keys_of_the_smallest_scale(dim, new):
    """Keys whose blocks all have scale code 0, 2^-127, and queries large enough for them to matter; keys of zeros between them."""
    def edit(k, v):
        k *= 2.0 ** -127
        k[3::5] = 0
        k[100:120, :, :32] = 0
    c = Chunk([250, 0], [new, 17], 2, 4, dim, 16, "bf16", seed=new, edit=edit)
    assert (c.cache.tensors[1][: 2 * (dim // 32)] != 255).any()
    c.q = (c.q.float().clamp(-3.9, 3.9) * 2.0 ** 125).to(torch.bfloat16)
    out, lse = c.run(scale=0.75)
    c.check(out, lse, scale=0.75)
    assert lse.max() - lse.min() > 1  # (the keys do matter)
