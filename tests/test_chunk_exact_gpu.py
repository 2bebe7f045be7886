"""Bits and range of the attention of several new tokens: what its logits, probabilities and keys have to hold at the ends of what
its description allows. Tolerances as in test_chunk_gpu, but for what a test says itself."""
import numpy as np
import pytest
import torch

from .test_chunk_gpu import Chunk
from .test_kv4_gpu import ROUND

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


def _against(c, out, floor, window=0):
    """Outputs to 16 bits of every probability: its first term is cut after 8 bits, which leaves less than 2^-7 of it, and the second
    term rounds that to 8 bits, so the two are off by 2^-16 of it at most. The logits are single products here, exact but for the
    factor's two roundings and the one in FP32, and below 8: 2^-20 with the exponential's own 2^-21; 2^-19 for the joins; the sums over
    n keys (n / 16 + 32) 2^-23. Then the output's rounding and `floor`, its smallest step."""
    D = c.cache.dim
    q, o = (t.double().cpu().numpy() for t in (c.q, out))
    for s, (b, n) in enumerate(zip(c.before, c.new)):
        k, v = c.of(s)
        pos, key = np.arange(b, b + n)[:, None], np.arange(b + n)[None]
        seen = (key <= pos) & ((key > pos - window) if window else True)
        for h in range(q.shape[1]):
            z = np.where(seen, q[c.rows[s]:c.rows[s + 1], h] @ k[:, h // c.group].T * float(np.float32(D ** -0.5)), -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            want, mag = p @ v[:, h // c.group], p @ np.abs(v[:, h // c.group])
            assert np.abs(z[seen]).max() < 8
            tol = (2.0 ** -16 + 2.0 ** -20 + 2.0 ** -19 + ((b + n) / 16 + 32) * 2.0 ** -23) * mag + ROUND[c.kind] * 1.01 * np.abs(want) + floor
            off = np.abs(o[c.rows[s]:c.rows[s + 1], h] - want)
            assert (off <= tol).all(), (s, h, (off / tol).max())
            # probabilities of 12 bits would not pass, where they are few (many average their errors)
            step = 2.0 ** (np.floor(np.log2(p, where=p > 0, out=np.zeros_like(p))) - 11)
            rough = (np.floor(p / step) * step) @ v[:, h // c.group]
            few = seen.sum(1) <= 12
            assert not few.any() or (np.abs(rough - want) > 2 * tol)[few].any()


@pytest.mark.parametrize("dim,group,before,new,window", [
    (64, 1, [2, 0], [40, 30], 0), (128, 3, [2, 30], [90, 60], 0), (128, 1, [500], [300], 0), (256, 2, [2, 100], [70, 33], 0), (128, 2, [3000], [25], 40)])
def test_probabilities_have_16_bits(dim, group, before, new, window):
    """Values that nearly cancel, so that what is left is small beside the output's own rounding of the terms: few keys of nearly
    equal weight, with logits from one element of q and k alone."""
    def edit(k, v):
        k[..., 1:] = 0
        k[..., 0] = np.float32([1, -0.5, 2, 1.5, -1, 0.5, 3])[np.arange(len(k)) % 7][:, None]
        v[:] = np.sign(v) * np.float32([1, 1.5, 2, 3])[np.arange(v.shape[-1]) % 4]
        v[1::2] = -v[::2][: len(v[1::2])]
    c = Chunk(before, new, 2, group, dim, 16, "f16", seed=dim, edit=edit)
    c.q[..., 1:] = 0
    c.q[..., 0] = (c.q[..., 0].float().abs().clamp(0.1, 2.0) * dim ** 0.5 / 8).half()
    out, _ = c.run(window=window)
    _against(c, out, 2.0 ** -25, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_next_to_the_smallest(dim):
    """V with scale codes from 0 to 8: sums where FP32 has fewer bits, outputs where BF16 has."""
    def edit(k, v):
        k[..., 1:] = 0
        v *= 2.0 ** -122
        v[::3, :, :32] *= 2.0 ** -5
    c = Chunk([150, 3], [60, 20], 2, 2, dim, 16, "bf16", seed=dim, edit=edit)
    c.q[..., 0] = c.q[..., 0].float().clamp(-1, 1).to(torch.bfloat16)
    out, _ = c.run()
    D = dim
    q, o = (t.double().cpu().numpy() for t in (c.q, out))
    for s, (b, n) in enumerate(zip(c.before, c.new)):
        k, v = c.of(s)
        seen = np.arange(b + n)[None] <= np.arange(b, b + n)[:, None]
        for h in range(4):
            z = np.where(seen, q[c.rows[s]:c.rows[s + 1], h] @ k[:, h // 2].T * D ** -0.5, -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            want, mag = p @ v[:, h // 2], p @ np.abs(v[:, h // 2])
            # BF16's smallest step is 2^-133: half of it for the output's rounding, as much for the terms' and sums' in FP32's last ones
            tol = (2.0 ** -15 + 40 * 2.0 ** -23) * mag + ROUND["bf16"] * 1.01 * np.abs(want) + 2.0 ** -133
            assert (np.abs(o[c.rows[s]:c.rows[s + 1], h] - want) <= tol).all(), (s, h)
