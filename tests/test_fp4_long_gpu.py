"""Projections with long rows: fewer tokens at a time above 8192 and 16384 columns, the streaming kernel above 32768,
and columns in chunks over many row tiles. Tolerances as in test_fp4_gpu.py."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref
from .test_fp4_gpu import TYPES, _close, _weights, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xk,yk", [("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("N,K,B", [
    (130, 8192, 64), (130, 8192 + 32, 33), (257, 9216, 64), (40, 16384, 72), (257, 12288, 40),  # 64 and 32 at a time
    (130, 16384 + 32, 17), (257, 20480, 33), (40, 32768, 64),                                     # 16 at a time
    (130, 32768 + 32, 9), (40, 65536, 20)])                                                       # 8, streamed
def test_long_rows_of_many_tokens(N, K, B, xk, yk):
    rng = np.random.default_rng(N + K + B)
    w, w64, *_ = _weights(rng, N, K)
    x = _x(rng, B, K, xk, pad=8)
    wide = torch.full((B, N + 3), 7.0, dtype=TYPES[yk], device="cuda")
    block_ops.wd_fp4_matvec(w, x, wide[:, :N])
    _close(wide[:, :N], x, w64, yk)
    assert (wide[:, N:] == 7.0).all()


@pytest.mark.parametrize("N,K,B", [(80003, 13312, 3), (80003, 16416, 9), (5003, 65536, 8), (20003, 16384, 40)])
def test_long_rows_over_many_row_tiles(N, K, B):
    """More than 32 row tiles of a CTA with their columns in chunks; clusters of 8 in rounds. The rows repeat every 61."""
    rng = np.random.default_rng(N)
    base, scales = rng.integers(0, 16, (61, K), dtype=np.uint8), rng.integers(115, 130, (61, K // 32), dtype=np.uint8)
    at = torch.arange(N, device="cuda") % 61
    w = block_ops.Fp4Weights.from_codes(torch.from_numpy(ref.row_major_bytes(base)).cuda()[at], torch.from_numpy(scales).cuda()[at])
    x = _x(rng, B, K, "bf16")
    y = torch.full((B, N), float("nan"), device="cuda")
    block_ops.wd_fp4_matvec(w, x, y)
    w64 = ref.values(base, scales)
    for n in range(0, N, 61):
        part = y[:, n:n + 61]
        if n % (61 * 50) == 0 or n + 61 > N:
            _close(part, x, w64[:part.shape[1]], "f32")
    # the rest against the rows just checked: twice the tolerance lies between two right sums
    first = y[:, :61].double().cpu().numpy()
    mag = np.abs(x.double().cpu().numpy()) @ np.abs(w64).T
    tol = 2 * ((K / 16 + 32) * 2.0 ** -23 * mag + 2.0 ** -24 * 1.01 * np.abs(first)
               + 2.0 ** -40 * np.abs(x.double().cpu().numpy()).max(1)[:, None] * np.abs(w64).sum(1))
    whole = y[:, :N // 61 * 61].view(B, -1, 61).double()
    off = (whole - torch.from_numpy(first).cuda()[:, None]).abs()
    assert (off <= torch.from_numpy(tol).cuda()[:, None]).all()
