"""Attention over the 4-bit cache where its weights' bits and range show.

A weight p 2^s is two BF16 terms: off by at most 2^-17 of itself, and in FP32's range of exponents. The
exponentials and joins are off by 2^-20, the sum over keys by 2^-20 of the magnitudes, and a logit as in
test_kv4_gpu.py. No part of the tolerance is relative to the largest value of a block: every bound is of the
magnitudes that make up the output.
"""
import numpy as np
import pytest
import torch

from . import _block_ref as ref
from .test_kv4_gpu import ROUND, Filled, _attend, _q

pytestmark = pytest.mark.gpu


def _check_elements(f, q, out, kind):
    D = q.shape[2]
    for s in range(q.shape[0]):
        want, _, mag, reach = ref.attend(q[s].double().cpu().numpy(), *f.of(s), float(np.float32(D ** -0.5)))
        d = ((D / 32 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach[:, None]
        tol = (2 * d + 2.0 ** -17 + 2.0 ** -19) * mag + ROUND[kind] * 1.01 * np.abs(want) + (2.0 ** -25 if kind == "f16" else 2.0 ** -120)
        off = np.abs(out[s].double().cpu().numpy() - want)
        assert (off <= tol).all(), (s, (off / tol).max())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", [(64, 3), (64, 16), (128, 8), (128, 16), (256, 8)])
def test_sums_that_cancel(dim, group, kind):
    """Few keys of nearly equal probability: many outputs are small beside their terms, so they are rounded finely."""
    f = Filled([2, 3, 5, 40], 2, dim, 16, kind, seed=group)
    q = (_q(f.rng, 4, 2 * group, dim, kind) * 0.02).contiguous()
    out, _ = _attend(f, q)
    _check_elements(f, q, out, kind)


@pytest.mark.parametrize("dim,group", [(64, 1), (128, 8), (128, 16), (256, 8)])
@pytest.mark.parametrize("n,loud_at", [(50, 3), (50, 47), (5000, 2600)])
def test_a_loud_value_of_negligible_probability(n, loud_at, dim, group):
    """One key that no query wants holds values 2^40 times the others': they stay what they are."""
    def edit(k, v):
        k[:, :, 0] = 1.0
        k[loud_at, :, 0] = -512.0  # with the query's 20 below: e^-1000 or less
        v[loud_at] *= 2.0 ** 40
    f = Filled([n], 1, dim, 16, edit=edit)
    q = _q(f.rng, 1, group, dim).clone()
    q[:, :, 0] = 20.0
    out, _ = _attend(f, q)
    _check_elements(f, q, out, "bf16")


@pytest.mark.parametrize("dim,group", [(64, 1), (128, 8), (128, 16), (256, 8)])
@pytest.mark.parametrize("n", [40, 3000])
def test_outputs_that_only_improbable_keys_make(n, dim, group):
    """One key takes nearly all of the probability and holds zeros in half of the channels."""
    def edit(k, v):
        k[:, :, 0] = 0.0
        k[7, :, 0] = 16.0
        v[7, :, ::2] = 0.0
    f = Filled([n], 1, dim, 16, edit=edit)
    q = _q(f.rng, 1, group, dim).clone()
    q[:, :, 0] = 30.0
    out, _ = _attend(f, q)
    _check_elements(f, q, out, "bf16")


@pytest.mark.parametrize("dim,group", [(64, 3), (128, 8), (128, 16), (256, 8)])
def test_f16_queries_are_exact_beside_the_largest(dim, group):
    """The largest F16 query under zeros of K, the smallest subnormals under large keys."""
    def edit(k, v):
        k *= 2.0 ** 10
        k[:, :, :32] = 0
    f = Filled([40, 3000], 1, dim, 16, "f16", edit=edit)
    q = torch.from_numpy(f.rng.integers(-7, 8, (2, group, dim)).astype(np.float32) * 2.0 ** -24).half().cuda()
    q[:, :, 5] = 65504.0
    scale = 2.0 ** 14
    out, _ = _attend(f, q, scale=scale)
    for s in range(2):
        want, _, mag, reach = ref.attend(q[s].double().cpu().numpy(), *f.of(s), scale)
        d = ((dim / 32 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach[:, None]
        tol = (2 * d + 2.0 ** -17 + 2.0 ** -19) * mag + 2.0 ** -11 * 1.01 * np.abs(want) + 2.0 ** -25
        assert (np.abs(out[s].double().cpu().numpy() - want) <= tol).all()
