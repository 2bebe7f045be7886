"""Rotary positions on the GPU against their definition in 64 bits.

Tolerance, in units of 2^-24 times (|a| + |b|) |magnitude| of a pair: sine and cosine are
off by 2.5 (the angle 0.4 for its conversion, 0.8 and 0.4 for the product with 2 pi and its
rounding, the series 0.9), their product with the magnitude by 1.5 (its own rounding
among it), the products and sums of the pair by 2: 6. Then one rounding to the type.
The codes of the cache have to be those of the exact value.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -126}


def _n(t):
    return t.double().cpu().numpy()


def turned(x, pos, freqs, interleaved, magnitude=1.0):
    """x [T, heads, dim] turned, and |a| + |b| of every element's pair (0 where none)."""
    n = len(freqs)
    angle = np.asarray(pos, np.float64)[:, None] * freqs
    c, s = magnitude * np.cos(angle)[:, None], magnitude * np.sin(angle)[:, None]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    y, size = x.copy(), np.zeros_like(x)
    at = (np.s_[..., 0:2 * n:2], np.s_[..., 1:2 * n:2]) if interleaved else (np.s_[..., :n], np.s_[..., n:2 * n])
    y[at[0]], y[at[1]] = a * c - b * s, b * c + a * s
    size[at[0]] = size[at[1]] = np.abs(a) + np.abs(b)
    return y, size * abs(magnitude)


def _close(got, x, pos, freqs, interleaved, kind, magnitude=1.0):
    want, size = turned(_n(x), pos, freqs, interleaved, magnitude)
    tol = 6 * 2.0 ** -24 * size + ROUND[kind] * 1.001 * np.abs(want) + TINY[kind]
    off = np.abs(_n(got) - want)
    assert (off <= tol).all(), (off / tol).max()
    assert np.array_equal(_n(got)[..., 2 * len(freqs):], _n(x)[..., 2 * len(freqs):])


def _x(T, heads, dim, kind, pad=0, seed=0):
    wide = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, heads + pad, dim)).astype(np.float32))
    return wide.to(TYPES[kind]).cuda()[:, :heads]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,dim,rot,pad", [
    (1, 1, 16, 16, 0), (1, 36, 128, 128, 4), (3, 5, 24, 16, 0), (7, 3, 80, 32, 1), (129, 9, 96, 96, 0), (64, 40, 128, 64, 8),
    (700, 2, 256, 64, 3), (33, 1, 1024, 1024, 0), (5, 70, 256, 256, 0), (2000, 6, 64, 64, 0), (300, 1, 200, 144, 2)])
def test_shapes(T, heads, dim, rot, pad, interleaved, kind):
    freqs = block_ops.rope_freqs(rot)
    rope = block_ops.Rope(freqs, interleaved)
    x = _x(T, heads, dim, kind, pad, seed=T)
    pos = np.random.default_rng(T + 1).integers(0, 5000, T).astype(np.int32)
    p = torch.from_numpy(pos).cuda()
    out = torch.full((T, heads + 2, dim), 7.0, dtype=x.dtype, device="cuda")
    assert block_ops.wd_rope(rope, x, p, out[:, 1:-1]).data_ptr() == out[:, 1:-1].data_ptr()
    _close(out[:, 1:-1], x, pos, freqs.numpy(), interleaved, kind)
    assert (out[:, 0] == 7).all() and (out[:, -1] == 7).all()
    same = x.clone() if pad == 0 else x
    kept = x.clone()
    assert block_ops.wd_rope(rope, same, p) is same  # in place
    assert torch.equal(same, out[:, 1:-1])
    back = block_ops.wd_rope(rope, same.contiguous(), -p)  # negative positions turn back
    assert (np.abs(_n(back) - _n(kept)) <= 4 * (ROUND[kind] + 2.0 ** -21) * np.abs(_n(kept)).max()).all()


@pytest.mark.parametrize("magnitude", [1.0, 1.3, 0.25, -1.0, 0.0])
@pytest.mark.parametrize("first", [0, 1, 131072, 2 ** 24 + 1, 2 ** 31 - 40, -(2 ** 31)])
def test_far_positions_and_magnitudes(first, magnitude):
    """Angles of millions of turns are as exact as those of the first. (pos * f in 64 bits is off by 2^-53 of itself: 2^-22.)"""
    freqs = block_ops.rope_freqs(128, base=500000.0, scaling="parts", factor=4.0, trained=8192)
    rope = block_ops.Rope(freqs, magnitude=magnitude)
    pos = np.arange(first, first + 40).astype(np.int32)
    x = _x(40, 3, 128, "f32", seed=5)
    out = block_ops.wd_rope(rope, x, torch.from_numpy(pos).cuda(), torch.empty_like(x))
    want, size = turned(_n(x), pos, freqs.numpy(), False, magnitude)
    slack = 2.0 ** -53 * abs(float(first)) * 2 + 6 * 2.0 ** -24
    assert (np.abs(_n(out) - want) <= slack * size + 2.0 ** -24 * np.abs(want)).all()


def test_special_values():
    freqs = block_ops.rope_freqs(16)
    rope = block_ops.Rope(freqs)
    x = _x(2, 2, 32, "f32")
    x[0, 0, 3], x[0, 1, 20], x[1, 0, 12] = float("nan"), float("inf"), float("inf")
    out = block_ops.wd_rope(rope, x, torch.tensor([5, 9], dtype=torch.int32, device="cuda"), torch.empty_like(x))
    bad = torch.zeros(2, 2, 32, dtype=torch.bool)
    bad[0, 0, [3, 11]] = bad[0, 1, 20] = bad[1, 0, [4, 12]] = True  # pairs (3, 11) and (4, 12); 20 does not turn
    assert torch.equal(~torch.isfinite(out).cpu(), bad)
    assert torch.isinf(out[0, 1, 20])


def _fill(news, before, heads, q_heads, dim, page, kind, seed=0, edit=None, extra=0):
    rng = np.random.default_rng(seed)
    per = [-(-(a + b) // page) for a, b in zip(before, news)]
    pages = rng.permutation(sum(per) + 2).astype(np.int32)
    table = np.full((len(news), max(per + [1])), -1, np.int32)
    for i, n in enumerate(per):
        table[i, :n] = pages[sum(per[:i]):sum(per[:i]) + n]
    cache = block_ops.Kv4Cache(sum(per) + 2, page, heads, dim)
    for t in cache.tensors:
        t.fill_(255)
    T = sum(news) + extra
    qkv = (rng.standard_normal((T, q_heads + 2 * heads, dim)) * (1 + 5 * (rng.random((1, 1, dim)) < 0.05))).astype(np.float32)
    if edit:
        edit(qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:])
    qkv = torch.from_numpy(qkv).to(TYPES[kind]).cuda()
    q, k, v = qkv.split([q_heads, heads, heads], 1)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    lens = torch.tensor(before, dtype=torch.int32, device="cuda")
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, news)] + [np.zeros(0, int)])
    return cache, torch.from_numpy(table).cuda(), lens, cu, q, k, v, pos


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("news,before,heads,q_heads,dim,rot,interleaved,page", [
    ([1], [0], 1, 1, 64, 64, False, 16), ([1, 1, 1], [5, 16, 33], 2, 6, 128, 128, False, 16), ([5, 0, 33, 16], [0, 7, 1, 100], 2, 8, 128, 64, True, 16),
    ([70, 1, 64], [3, 0, 2], 3, 3, 256, 256, True, 32), ([300, 129], [0, 1], 1, 16, 128, 32, False, 128), ([2000], [7], 2, 10, 64, 16, False, 256),
    ([63, 65], [100000, 31], 2, 40, 128, 128, False, 64), ([31, 18], [1, 0], 17, 17, 64, 48, False, 16), ([400, 177], [9, 30], 9, 18, 256, 96, True, 32)])
def test_append_holds_the_nearest_to_the_exact_turn(news, before, heads, q_heads, dim, rot, interleaved, page, kind):
    cache, table, lens, cu, q, k, v, pos = _fill(news, before, heads, q_heads, dim, page, kind, seed=dim + len(news))
    freqs = block_ops.rope_freqs(rot)
    rope = block_ops.Rope(freqs, interleaved)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    kept = [t.clone() for t in (q, k, v)]
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, q_out, cu, err)
    assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(kept, (q, k, v)))
    _close(q_out, q, pos, freqs.numpy(), interleaved, kind)
    got_k, got_v = (torch.empty(k.shape, device="cuda") for _ in range(2))
    block_ops.wd_kv4_gather(cache, table, lens, got_k, got_v, cu, err)
    want, _ = turned(_n(k), pos, freqs.numpy(), interleaved)
    assert np.array_equal(_n(got_v), ref.rounded(_n(v)))
    assert np.array_equal(_n(got_k), ref.rounded(want))
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, cu_new=cu)  # in place
    assert torch.equal(q, q_out)
    if max(news) == 1:
        block_ops.wd_kv4_rope_append(cache, rope, kept[0], k, v, table, lens)  # without cu_new: one each
        assert torch.equal(kept[0], q_out)


@pytest.mark.parametrize("interleaved", [False, True])
def test_many_codes_are_all_exact(interleaved):
    """Millions of elements, so that FP32's own rounding would put some on the wrong side of a border."""
    cache, table, lens, cu, q, k, v, pos = _fill([9000, 3001], [17, 4], 4, 4, 128, 64, "bf16", seed=3)
    freqs = block_ops.rope_freqs(128)
    block_ops.wd_kv4_rope_append(cache, block_ops.Rope(freqs, interleaved, 1.1), q, k, v, table, lens, cu_new=cu)
    got_k, got_v = (torch.empty(k.shape, device="cuda") for _ in range(2))
    block_ops.wd_kv4_gather(cache, table, lens, got_k, got_v, cu)
    for first in range(0, 12001, 3000):
        at = slice(first, first + 3000)
        assert np.array_equal(_n(got_k[at]), ref.rounded(turned(_n(k[at]), pos[at], freqs.numpy(), interleaved, 1.1)[0]))


def test_borders_and_special_blocks():
    """Values on the borders themselves (position 0 turns by nothing), cancelling pairs, zeros, infinities and NaN."""
    def edit(k, v):
        k[0, 0, :32] = [7.9, 5, 2.5, 0.25, 0.75, 1.25, 1.75, 3.5] * 4
        k[0, 0, 32:64] = [-7.9, -5, -2.5, -0.25, -0.75, -1.25, -1.75, -3.5] * 4
        k[0, 1] = 4.0
        k[1] = 0
        k[2, 0, 3], k[3, 1, 70], v[2, 0, 40] = np.inf, np.nan, np.nan
        k[4] *= 1e-25
        k[5] *= 1e25
    cache, table, lens, cu, q, k, v, pos = _fill([9], [0], 2, 2, 128, 16, "bf16", edit=edit)
    freqs = block_ops.rope_freqs(64)
    block_ops.wd_kv4_rope_append(cache, block_ops.Rope(freqs), q, k, v, table, lens, cu_new=cu)
    got_k, got_v = (torch.empty(k.shape, device="cuda") for _ in range(2))
    block_ops.wd_kv4_gather(cache, table, lens, got_k, got_v, cu)
    with np.errstate(invalid="ignore"):
        want = turned(_n(k), pos, freqs.numpy(), False)[0]
    assert np.array_equal(_n(got_k), ref.rounded(want), equal_nan=True)
    assert np.array_equal(_n(got_v), ref.rounded(_n(v)), equal_nan=True)
    assert np.isnan(_n(got_k)[2, 0, :64]).all() and np.isnan(_n(got_k)[3, 1, 64:96]).all()


@pytest.mark.parametrize("steps", [[1] * 9, [3, 1, 4, 1], [2, 7]])
def test_steps_and_one_call_hold_the_same(steps):
    freqs = block_ops.rope_freqs(128)
    rope = block_ops.Rope(freqs)
    cache, table, lens, cu, q, k, v, pos = _fill([9, 9], [0, 3], 2, 4, 128, 16, "f16", seed=1)
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, torch.empty_like(q), cu)
    whole = [t.clone() for t in cache.tensors]
    for t in cache.tensors:
        t.fill_(255)
    at = 0
    for n in steps:
        rows = torch.cat([torch.arange(at, at + n), torch.arange(9 + at, 9 + at + n)]).cuda()
        c = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
        block_ops.wd_kv4_rope_append(cache, rope, q[rows], k[rows], v[rows], table, lens + at, cu_new=c)
        at += n
    assert all(torch.equal(a, b) for a, b in zip(whole, cache.tensors))


def test_rows_without_a_place():
    """Padding stays as it was; a token without a page is flagged and left out, its query turned all the same."""
    rope = block_ops.Rope(block_ops.rope_freqs(64))
    cache, table, lens, cu, q, k, v, pos = _fill([3, 2], [0, 14], 1, 2, 64, 16, "bf16", extra=4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, q_out, cu, err)
    assert int(err) == 0 and (q_out[5:] == 9).all()
    _close(q_out[:5], q[:5], pos, block_ops.rope_freqs(64).numpy(), False, "bf16")
    before = [t.clone() for t in cache.tensors]
    table[0, 0] = cache.pages
    again = torch.full_like(q_out, 9.0)
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, again, cu, err)
    assert int(err) == 1 and torch.equal(again, q_out) and all(torch.equal(a, b) for a, b in zip(before, cache.tensors))
    err.zero_()
    again.fill_(9)
    lens[1] = -3
    table[0, 0] = 1 << 30
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, again, cu, err)
    assert int(err) == 1 and (again[3:] == 9).all() and torch.equal(again[:3], q_out[:3])
    assert all(torch.equal(a, b) for a, b in zip(before, cache.tensors))


def test_another_stream_and_a_graph():
    rope = block_ops.Rope(block_ops.rope_freqs(128))
    cache, table, lens, cu, q, k, v, pos = _fill([1] * 6, [4, 9, 0, 31, 77, 15], 2, 8, 128, 16, "bf16")
    want = block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, torch.empty_like(q))
    held = [t.clone() for t in cache.tensors]
    p = torch.arange(6, dtype=torch.int32, device="cuda")
    alone = block_ops.wd_rope(rope, q, p, torch.empty_like(q))
    torch.cuda.synchronize()
    side, out, out2 = torch.cuda.Stream(), torch.zeros_like(want), torch.zeros_like(want)
    for t in cache.tensors:
        t.fill_(255)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, out)
        block_ops.wd_rope(rope, q, p, out2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(out2, alone) and all(torch.equal(a, b) for a, b in zip(held, cache.tensors))
    out.zero_()
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_refusals():
    rope = block_ops.Rope(block_ops.rope_freqs(64))
    x = _x(3, 2, 64, "bf16")
    p = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert block_ops.wd_rope(rope, x[:0], p[:0]).shape == (0, 2, 64)
    with pytest.raises(TypeError):
        block_ops.wd_rope(rope, x, p, x.float())
    with pytest.raises(TypeError):
        block_ops.wd_rope(rope, x, p.long())
    with pytest.raises(ValueError):
        block_ops.wd_rope(rope, x, p[:2])
    with pytest.raises(block_ops.WarpDecodeError, match="rot_dim"):
        block_ops.wd_rope(rope, x[..., :32].contiguous(), p)
    with pytest.raises(block_ops.WarpDecodeError, match="16 bytes"):
        block_ops.wd_rope(rope, torch.empty(3 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 2, 64), p)
    cache, table, lens, cu, q, k, v, pos = _fill([3], [0], 1, 2, 64, 16, "bf16")
    with pytest.raises(TypeError, match="one dtype"):
        block_ops.wd_kv4_rope_append(cache, rope, q.half(), k, v, table, lens, cu_new=cu)
    with pytest.raises(block_ops.WarpDecodeError, match="rot_dim"):
        block_ops.wd_kv4_rope_append(cache, block_ops.Rope(block_ops.rope_freqs(128)), q, k, v, table, lens, cu_new=cu)
    with pytest.raises(block_ops.WarpDecodeError):
        block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens)  # three rows, one sequence
