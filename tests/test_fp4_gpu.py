"""4-bit projections on the GPU against their definition in 64 bits.

Tolerance of a matvec output, for any order of the sums: the products are exact,
a sum of K of them passes at most K/16 + 32 FP32 additions in a row (MMAs of 16
products, scale blocks, warps, staged parts), each off by at most 2^-23 of the
magnitudes that it has summed; a value of x below 2^-32 of its token's largest is
off by 2^-40 of that; one rounding to the output's type at the end.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": (2.0 ** -24, 0.0), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def _weights(rng, N, K):
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = rng.integers(115, 130, (N, K // 32), dtype=np.uint8)
    w = block_ops.Fp4Weights.from_codes(torch.from_numpy(ref.row_major_bytes(codes)).cuda(),
                                        torch.from_numpy(scales).cuda())
    return w, ref.values(codes, scales), codes, scales


def _x(rng, B, K, kind, pad=0):
    x = np.zeros((B, K + pad), np.float32)
    x[:, :K] = rng.standard_normal((B, K)) * np.exp2(rng.integers(-6, 7, (B, 1)))
    wide = torch.from_numpy(x).to(TYPES[kind]).cuda()
    return wide[:, :K]


def _close(y, x, w, kind):
    x64 = x.double().cpu().numpy()
    want, mag = x64 @ w.T, np.abs(x64) @ np.abs(w).T
    K = w.shape[1]
    rel, least = ROUND[kind]
    tol = (K / 16 + 32) * 2.0 ** -23 * mag + 2.0 ** -40 * np.abs(x64).max(1)[:, None] * np.abs(w).sum(1) \
        + rel * np.abs(want) * 1.01 + least
    off = np.abs(y.double().cpu().numpy() - want)
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("N,K", [(1, 32), (16, 128), (17, 160), (130, 4096 + 96), (250, 9216)])
def test_pack_codes_is_the_documented_layout(N, K):
    w, _, codes, scales = _weights(np.random.default_rng(N), N, K)
    pc, ps = ref.pack_rows(codes, scales)
    assert np.array_equal(w.codes.cpu().numpy(), pc) and np.array_equal(w.scales.cpu().numpy(), ps)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_quantize_is_the_documented_rule(kind):
    rng = np.random.default_rng(5)
    v = (rng.standard_normal((37, 352)) * np.exp2(rng.integers(-12, 12, (37, 1)))).astype(np.float32)
    v[0, :32] = 0
    v[1, :32] = 1e-38  # subnormal block scale
    v[2, 3], v[3, 40], v[4, 70] = np.inf, np.nan, -np.inf
    v[5, :32] = np.array([8, 7, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -5, -0.0] + [0] * 20) * 2.0 ** -3
    v[6, :32] = 3e38 if kind != "f16" else 6e4
    wide = torch.zeros(37, 352 + 9, dtype=TYPES[kind], device="cuda")
    wide[:, :352] = torch.from_numpy(v).to(TYPES[kind])
    held = wide[:, :352].double().cpu().numpy()
    w = block_ops.Fp4Weights.quantize(wide[:, :352])
    codes, scales = ref.quantise(held)
    pc, ps = ref.pack_rows(codes, scales)
    assert np.array_equal(w.scales.cpu().numpy(), ps)
    got, want = w.codes.cpu().numpy(), pc
    # the codes of NaN blocks and the sign of a zero have no value of their own
    differ = np.flatnonzero(got != want)
    by_row = ps.reshape(-1, 8, 2, 4).swapaxes(1, 2).reshape(-1, 16, 1, 4, 1)
    keep = np.repeat(by_row == 255, 4, 2).repeat(4, 4).reshape(-1)
    nibbles = lambda a: np.stack([a & 15, a >> 4])  # noqa: E731
    g, h = nibbles(got[differ]), nibbles(want[differ])
    same = (g == h) | ((g & 7 == 0) & (h & 7 == 0))
    assert (same.all(0) | keep[differ]).all()


@pytest.mark.parametrize("B", [1, 2, 7, 8, 9, 16, 17, 24, 33, 64, 65, 130])
def test_tokens(B):
    rng = np.random.default_rng(B)
    w, w64, *_ = _weights(rng, 272, 512)
    x = _x(rng, B, 512, "bf16")
    y = torch.full((B, 272), float("nan"), device="cuda")
    assert block_ops.wd_fp4_matvec(w, x, y) is y
    _close(y, x, w64, "f32")


@pytest.mark.parametrize("xk", ["bf16", "f16"])
@pytest.mark.parametrize("yk", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,K,B", [(1, 32, 1), (33, 16416, 3), (33, 96, 3), (1003, 4128, 5), (129, 8192 + 64, 20), (515, 320, 40)])
def test_shapes_types_and_strides(N, K, B, xk, yk):
    rng = np.random.default_rng(N + K + B)
    w, w64, *_ = _weights(rng, N, K)
    w64 = w64 * 2.0 ** -6 if yk == "f16" else w64
    if yk == "f16":  # keep the sums inside f16's range
        codes, scales = ref.quantise(w64)
        w = block_ops.Fp4Weights.from_codes(torch.from_numpy(ref.row_major_bytes(codes)).cuda(),
                                            torch.from_numpy(scales).cuda())
        w64 = ref.values(codes, scales)
    x = _x(rng, B, K, xk, pad=24)
    wide = torch.full((B, N + 5), 7.0, dtype=TYPES[yk], device="cuda")
    block_ops.wd_fp4_matvec(w, x, wide[:, :N])
    _close(wide[:, :N], x, w64, yk)
    assert (wide[:, N:] == 7.0).all()  # nothing beside the rows is written


@pytest.mark.parametrize("yk", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,B", [(40003, 160, 8), (40003, 96, 16), (24001, 1152, 40)])
def test_many_rows(N, K, B, yk):
    """More rows than the CTAs take at a time: written as they end, in rounds, in rounds of clusters."""
    rng = np.random.default_rng(N + B)
    w, w64, *_ = _weights(rng, N, K)
    x = _x(rng, B, K, "bf16")
    wide = torch.full((B, N + 3), 7.0, dtype=TYPES[yk], device="cuda")
    block_ops.wd_fp4_matvec(w, x, wide[:, :N])
    _close(wide[:, :N], x, w64, yk)
    assert (wide[:, N:] == 7.0).all()


@pytest.mark.parametrize("N,K,B", [(12001, 4096, 40), (6001, 8192, 64)])
def test_rounds_of_wide_clusters(N, K, B):
    """More row tiles than clusters of 4 and of 8 CTAs take at a time."""
    rng = np.random.default_rng(N)
    w, w64, *_ = _weights(rng, N, K)
    x = _x(rng, B, K, "bf16")
    y = torch.full((B, N), float("nan"), device="cuda")
    block_ops.wd_fp4_matvec(w, x, y)
    _close(y, x, w64, "f32")
    again = torch.empty_like(y)
    block_ops.wd_fp4_matvec(w, x, again)
    assert torch.equal(y, again)


@pytest.mark.parametrize("B", [1, 12, 40])
def test_extremes(B):
    """Zero tokens, loud channels, infinities and NaN stay where they belong; scale codes 0, 254 and 255."""
    rng = np.random.default_rng(B)
    N, K = 48, 4096 + 128
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = np.full((N, K // 32), 120, np.uint8)
    scales[3, 5], scales[4], scales[7, 2] = 255, 0, 0
    w = block_ops.Fp4Weights.from_codes(torch.from_numpy(ref.row_major_bytes(codes)).cuda(),
                                        torch.from_numpy(scales).cuda())
    w64 = ref.values(codes, scales)
    x = _x(rng, B, K, "bf16").clone()
    x[0, 17] = 30000.0
    if B > 4:
        x[1] = 0
        x[2, 100] = float("inf")
        x[3, 4100] = float("nan")
        x[4] *= 2.0 ** -120
    y = torch.empty(B, N, device="cuda")
    block_ops.wd_fp4_matvec(w, x, y)
    got, x64 = y.double().cpu().numpy(), x.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = np.array([[np.sum(x64[b] * w64[n]) for n in range(N)] for b in range(B)])
        mag = np.array([[np.sum(np.abs(x64[b] * w64[n])) for n in range(N)] for b in range(B)])
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    fine = np.isfinite(want)
    tol = (K / 16 + 34) * 2.0 ** -23 * mag + 2.0 ** -40 * np.abs(x64).max(1)[:, None] * np.abs(w64).sum(1) + 2.0 ** -140
    assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all()
    if B > 4:
        assert (got[1][~np.isnan(want[1])] == 0).all()


@pytest.mark.parametrize("B", [1, 16, 48])
def test_same_result_on_every_call_and_on_another_stream(B):
    rng = np.random.default_rng(1)
    w, *_ = _weights(rng, 2048, 2048)
    x = _x(rng, B, 2048, "bf16")
    y0 = block_ops.wd_fp4_matvec(w, x, torch.empty(B, 2048, device="cuda")).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1 = torch.empty(B, 2048, device="cuda")
    torch.cuda.synchronize()
    block_ops.wd_fp4_matvec(w, x, y1, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        y2 = block_ops.wd_fp4_matvec(w, x, torch.empty(B, 2048, device="cuda"))
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2)


def test_empty_batch_and_refusals():
    w, *_ = _weights(np.random.default_rng(2), 32, 64)
    y = torch.empty(0, 32, device="cuda")
    block_ops.wd_fp4_matvec(w, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), y)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="expected shape"):
        block_ops.wd_fp4_matvec(w, x, torch.empty(2, 31, device="cuda"))
    with pytest.raises(block_ops.WarpDecodeError) as e:
        block_ops.wd_fp4_matvec(w, x.float(), torch.empty(2, 32, device="cuda"))
    assert e.value.status == 5
    with pytest.raises(ValueError, match="unsupported shape"):
        block_ops.Fp4Weights(16, 40)
