"""wd_kv4_attend with a scale of 0: logits of 0 whatever the keys, so every key weighs the same. Tolerance: 2^-15 of the magnitudes
for the weights' 16 bits and the FP32 sums over a few hundred keys, and the rounding of the output."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from .test_kv4_gpu import ROUND, Filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group", [(64, 2), (128, 8), (128, 16), (256, 3)])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_no_scale_with_large_keys(scale, dim, group):
    def edit(k, v):
        k[:] = 2.0 ** 99
        k[::2] *= -1
        v[::2] = np.abs(v[::2])
    lens = [300, 1, 40]
    f = Filled(lens, 2, dim, 16, edit=edit)
    q = torch.ones(3, 2 * group, dim, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    block_ops.wd_kv4_attend(f.cache, q, f.table_d, f.lens_d, out, block_ops.kv4_workspace(f.cache, 3, 2 * group), lse=lse, scale=scale)
    for s, n in enumerate(lens):
        v = np.repeat(f.of(s)[1], group, 1)
        want, mag = v.mean(0), np.abs(v).mean(0)
        off = np.abs(out[s].double().cpu().numpy() - want)
        assert (off <= 2.0 ** -15 * mag + ROUND["bf16"] * 1.01 * np.abs(want)).all()
        assert (np.abs(lse[s].double().cpu().numpy() - np.log(n)) <= 2.0 ** -18).all()
