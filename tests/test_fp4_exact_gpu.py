"""4-bit projections whose scales and values are far apart, against their definition in 64 bits.

No part of the tolerance is relative to what a row or a token holds elsewhere: x is exact here (its values lie
within 2^20 of one another), so an output is off by the roundings of its own sum, as in test_fp4_gpu.py, and by FP32's
smallest values.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref
from .test_fp4_gpu import TYPES

pytestmark = pytest.mark.gpu


def _run(codes, scales, x):
    w = block_ops.Fp4Weights.from_codes(torch.from_numpy(ref.row_major_bytes(codes)).cuda(), torch.from_numpy(scales).cuda())
    y = torch.full((x.shape[0], codes.shape[0]), 5.0, device="cuda")
    block_ops.wd_fp4_matvec(w, x, y)
    return y.double().cpu().numpy(), ref.values(codes, scales)


def _check(got, x, w64):
    x64 = x.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        terms = [x64[b] * w64 for b in range(x64.shape[0])]  # (a product of zero and infinity is NaN, as it is in a sum)
        want, mag = np.stack([t.sum(1) for t in terms]), np.stack([np.abs(t).sum(1) for t in terms])
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want) & (np.abs(want) < 2.0 ** 127)
    beyond = np.abs(want) >= 2.0 ** 128
    assert np.array_equal(got[beyond], np.copysign(np.inf, want[beyond]))
    off, tol = np.abs(got[fine] - want[fine]), (w64.shape[1] / 16 + 34) * 2.0 ** -23 * mag[fine] + 2.0 ** -140
    assert (off <= tol).all(), (off / tol).max()


def _x(rng, B, K, kind="bf16"):
    return torch.from_numpy(rng.uniform(0.5, 2.0, (B, K)).astype(np.float32) * rng.choice([-1, 1], (B, K))).to(TYPES[kind]).cuda()


SIZES = [(40, 256, 9), (300, 4096, 9), (130, 4128, 40), (515, 512, 64), (5000, 160, 17), (33, 352, 130)]
BATCHES = [(40, 256, 8), (300, 4096, 1), *SIZES]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,B", BATCHES)
def test_zeros_may_have_any_scale(N, K, B, kind):
    """A block of zeros with a scale far above the row's others."""
    rng = np.random.default_rng(N + B)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = rng.integers(100, 104, (N, K // 32), dtype=np.uint8)
    at = rng.integers(0, K // 32, N)
    for n in range(0, N, 3):
        codes[n, 32 * at[n]:32 * at[n] + 32] = rng.integers(0, 2, 32) * 8  # zeros of either sign
        scales[n, at[n]] = 180
    x = _x(rng, B, K, kind)
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,B", BATCHES)
def test_zeros_of_x_under_the_loudest_blocks(N, K, B, kind):
    """What x does not reach must not take the precision of what it does."""
    rng = np.random.default_rng(N + B)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = rng.integers(100, 104, (N, K // 32), dtype=np.uint8)
    scales[:, 2] = 180
    scales[::5, 1] = 150
    x = _x(rng, B, K, kind)
    x[:, 32:96] = 0
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,B", BATCHES)
def test_scales_on_both_sides_of_what_f16_holds(N, K, B, kind):
    """One loud block to a row under which some tokens are 0; the others 2^-24 to 2^-60 of it."""
    rng = np.random.default_rng(N + B)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = (160 - rng.choice([24, 25, 26, 27, 28, 40, 60], (N, K // 32))).astype(np.uint8)
    at = rng.integers(0, 2, N)
    scales[np.arange(N), at] = 160
    x = _x(rng, B, K, kind)
    x[::2, :64] = 0
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)


@pytest.mark.parametrize("N,K,B", BATCHES)
def test_any_scales(N, K, B):
    rng = np.random.default_rng(N + B)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    codes[:, rng.random(K) < 0.5] = 0
    scales = rng.integers(30, 200, (N, K // 32), dtype=np.uint8)
    x = _x(rng, B, K)
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)


@pytest.mark.parametrize("N,K,B", SIZES)
def test_an_infinity_meets_a_quiet_block(N, K, B):
    """The products of an infinity are infinite, NaN where a code is 0, whatever the scale."""
    rng = np.random.default_rng(N + B)
    codes = rng.integers(1, 8, (N, K), dtype=np.uint8)
    codes[::4, 40] = 0
    scales = np.full((N, K // 32), 100, np.uint8)
    scales[:, 3] = 180
    x = _x(rng, B, K)
    x[1, 40] = float("inf")
    x[3, 41] = -float("inf")
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,B", [(40, 256, 1), (40, 256, 8), (300, 4096, 5), (40003, 160, 8), (33, 16416, 3), (40, 256, 9), (300, 4096, 40)])
def test_the_largest_scales(N, K, B, kind):
    """Scale code 254: results that fit FP32, from small x, and infinities where they do not."""
    rng = np.random.default_rng(N + B)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = rng.integers(120, 255, (N, K // 32), dtype=np.uint8)
    scales[:, 0] = 254
    codes[N // 2:, :32] = 7  # one row in two ends at the last values of FP32 or beyond
    x = _x(rng, B, K, kind) * 2.0 ** -12
    x[0] = x[0].abs() * 2.0 ** 12
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)
    assert np.isfinite(got[1:]).all()


@pytest.mark.parametrize("N,K,B", [(300, 4096, 5), (40003, 160, 8), (33, 16416, 3), (300, 4096, 12)])
def test_infinities_and_nan_in_x(N, K, B):
    rng = np.random.default_rng(N + B)
    codes = rng.integers(1, 8, (N, K), dtype=np.uint8)
    codes[::4, 40] = 0
    scales = rng.integers(100, 104, (N, K // 32), dtype=np.uint8)
    scales[::5, 2] = 255
    x = _x(rng, B, K)
    x[1, 40] = float("inf")
    x[2, 41] = float("nan")
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)


@pytest.mark.parametrize("N,K,B", BATCHES)
def test_f16_values_are_exact_beside_the_largest(N, K, B):
    """The largest F16 values under zeros, the smallest subnormals under the rest."""
    rng = np.random.default_rng(N + B)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    codes[:, :8] = 0
    scales = rng.integers(120, 124, (N, K // 32), dtype=np.uint8)
    x = torch.from_numpy(rng.integers(-7, 8, (B, K)).astype(np.float32) * 2.0 ** -24).half().cuda()
    x[:, 3] = 65504.0
    x[1:, 5] = -32768.0
    got, w64 = _run(codes, scales, x)
    _check(got, x, w64)
