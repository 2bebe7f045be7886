"""Ends of the ranges of the operators for several new tokens: tables of one key tile, prompts cut at many places, keys with
scales of every range, and turned appends large enough for their prefetching form. Tolerances are those of the operators' own
tests: a block of a key 2^-36 below its largest counts as 0, at most 2^-30 of that key's sum |q k|, far below d there."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref
from .test_chunk_gpu import Chunk
from .test_decoder_layer_extend_gpu import layer  # noqa: F401
from .test_decoder_layer_gpu import layer as plain_layer  # noqa: F401
from .test_rope_gpu import _fill, turned

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before,new", [([0], [1]), ([0, 0, 0], [64, 1, 33]), ([63, 0, 31, 1], [1, 0, 32, 63]), ([100, 0, 127], [28, 128, 1])])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 3), (256, 5)])
def test_tables_of_one_tile(before, new, dim, group):
    """Items that are never split are not joined; a wider table, whose items could be, gives the same bits."""
    c = Chunk(before, new, 2, group, dim, 16, seed=dim)
    out, lse = c.run()
    c.check(out, lse)
    wide = torch.nn.functional.pad(c.table_d, (0, 24), value=-1)
    assert wide.shape[1] * 16 > 128
    again = c.run(table=wide)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    empty = torch.tensor([-1] * len(new), dtype=torch.int32, device="cuda")  # negative lengths: no key at all
    out, lse = c.run(start=empty)
    assert (out == 0).all() and torch.isinf(lse).all()


@pytest.mark.parametrize("dim,group,new,window", [(64, 5, 1500, 0), (128, 5, 1500, 0), (128, 16, 700, 300), (256, 3, 1100, 0), (256, 7, 900, 200)])
def test_prompts_cut_at_many_places(dim, group, new, window):
    c = Chunk([0, 77], [new, new // 3], 3, group, dim, 64, "f16", seed=group)
    out, lse = c.run(window=window)
    c.check(out, lse, window=window)
    again = c.run(window=window)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dim,new", [(64, 40), (128, 40), (128, 300), (256, 40)])
def test_keys_with_scales_of_every_range(dim, new):
    """Keys whose scales f16 takes, ones whose all or some do not, next to each other, in every mixture a run can have."""
    def edit(k, v):
        k[::6] *= 2.0 ** 13                # above
        k[1::6, :, :32] *= 2.0 ** -40      # a block below
        k[2::6] *= 2.0 ** -30              # all below
        k[3::24] = 0
        k[64:80] *= 2.0 ** -22             # a whole run near the lower end
        k[96:112, :, 32:64] *= 2.0 ** 20
    c = Chunk([250], [new], 2, 4, dim, 16, "bf16", seed=new, edit=edit)
    c.q = (c.q.float() * 2.0 ** -9).to(torch.bfloat16)
    c.check(*c.run())


@pytest.mark.parametrize("q_heads,heads,dim,rot,interleaved", [(33, 2, 128, 128, False), (5, 1, 256, 64, True), (64, 8, 64, 48, False)])
def test_a_long_turned_append_is_many_short_ones(q_heads, heads, dim, rot, interleaved):
    """The same bytes from one call and from calls of a few tokens, the queries as wd_rope turns them, nothing behind the last row."""
    news, extra = [2500, 0, 1601], 9
    cache, table, lens, cu, q, k, v, pos = _fill(news, [30, 4, 1], heads, q_heads, dim, 64, "bf16", seed=rot, extra=extra)
    rope = block_ops.Rope(block_ops.rope_freqs(rot), interleaved)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    block_ops.wd_kv4_rope_append(cache, rope, q, k, v, table, lens, out, cu)
    whole = [t.clone() for t in cache.tensors]
    T = sum(news)
    assert (out[T:] == 7).all()
    positions = torch.tensor(pos[:T], dtype=torch.int32, device="cuda")
    turned = block_ops.wd_rope(rope, q[:T], positions, torch.empty(q[:T].shape, dtype=q.dtype, device="cuda"))
    assert torch.equal(out[:T], turned)
    for t in cache.tensors:
        t.fill_(255)
    short = torch.empty_like(out)
    for first in range(0, 2500, 500):  # 500 tokens of the first sequence, then what is left of the last
        n, m = 500, (330 if first < 1500 else 611 if first == 1500 else 0)
        at = min(first // 500, 3) * 330
        rows = torch.cat([torch.arange(first, first + n), torch.arange(2500 + at, 2500 + at + m)]).cuda()
        c = torch.tensor([0, n, n, n + m], dtype=torch.int32, device="cuda")
        step = lens + torch.tensor([first, 0, at], dtype=torch.int32, device="cuda")
        short[rows] = block_ops.wd_kv4_rope_append(cache, rope, q[rows], k[rows], v[rows], table, step, cu_new=c)
    assert all(torch.equal(a, b) for a, b in zip(whole, cache.tensors)) and torch.equal(short[:T], out[:T])


@pytest.mark.parametrize("interleaved,magnitude", [(False, 1.0), (True, 1.0), (False, -1.0), (False, 1.25)])
def test_pairs_that_do_not_turn(interleaved, magnitude):
    """Frequencies of 0, and some so low that the first angles vanish in FP32 but not in 64 bits, where BF16 inputs often lie on a
    border between codes."""
    cache, table, lens, cu, q, k, v, pos = _fill([2000, 300], [0, 5], 3, 3, 128, 32, "bf16", seed=11)
    freqs = block_ops.rope_freqs(128)
    freqs[16:40] = 0.0
    freqs[40:] = torch.tensor([5e-11, -3e-11, 1e-12]).double().repeat(8)
    block_ops.wd_kv4_rope_append(cache, block_ops.Rope(freqs, interleaved, magnitude), q, k, v, table, lens, cu_new=cu)
    got = torch.empty(k.shape, device="cuda")
    block_ops.wd_kv4_gather(cache, table, lens, got, torch.empty_like(got), cu)
    want = turned(k.double().cpu().numpy(), pos, freqs.numpy(), interleaved, magnitude)[0]
    assert np.array_equal(got.double().cpu().numpy(), ref.rounded(want))


def test_padding_after_rows_of_nan(layer):  # noqa: F811
    """What an earlier call left in the layer's buffers reaches no padding row of a later one."""
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    start, err = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([3, 0], [0]))
    x = torch.randn(12, layer.w.moe.shape.H, device="cuda").to(torch.bfloat16)
    for t in layer.cache.tensors:
        t.zero_()
    bad = x.clone()
    bad[5:] = float("nan")
    layer.extend(bad, table, start, torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda"))
    for t in layer.cache.tensors:
        t.zero_()
    out = layer.extend(x.clone(), table, start, torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda"), err)
    assert int(err) == 0 and torch.isfinite(out.float()).all()
