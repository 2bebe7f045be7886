"""The 4-bit KV cache at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref
from .test_kv4_gpu import Filled, _attend, _q, _raw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 64, 2 ** 31 - 1])
@pytest.mark.parametrize("lens", [[5], [300, 0, 77], [9000, 40]])
def test_a_window_past_every_key_is_no_window(lens, window):
    f = Filled(lens, 2, 128, 16)
    q = _q(f.rng, len(lens), 16, 128)
    for a, b in zip(_attend(f, q, window=window), _attend(f, q)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [-1, 1 << 30])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 8), (128, 16), (256, 3)])
@pytest.mark.parametrize("lens", [[1], [64, 40], [20000, 33, 0, 700]])
def test_a_row_without_any_page_is_a_row_without_keys(lens, dim, group, bad):
    """Rows whole in a CTA and rows cut over many; their neighbours stay as they are."""
    f = Filled(lens, 1, dim, 16)
    q = _q(f.rng, len(lens), group, dim)
    table = f.table_d.clone()
    table[0] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _attend(f, q, table=table, err_flag=err)
    assert int(err) == 1
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    want, want_lse = _attend(f, q)
    assert torch.equal(out[1:], want[1:]) and torch.equal(lse[1:], want_lse[1:])


@pytest.mark.parametrize("window", [1, 40, 9000])
def test_a_window_that_reaches_no_page_has_no_keys(window):
    f = Filled([20000], 2, 128, 16)
    q = _q(f.rng, 1, 8, 128)
    table = f.table_d.clone()
    table[:, (20000 - window) // 16:] = -1
    out, lse = _attend(f, q, table=table, window=window)
    assert (out == 0).all() and (lse == -float("inf")).all()
    out, _ = _attend(f, q, table=table)  # the keys before it count without a window
    assert torch.isfinite(out).all() and (out != 0).any()


def _fresh(pages=4, page=16, heads=2, dim=128):
    cache = block_ops.Kv4Cache(pages, page, heads, dim)
    for t in cache.tensors:
        t.fill_(255)
    return cache


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("cuts", [[1], [3], [1, 2, 3, 4, 5], [5, 6, 11], [9, 23, 41, 57]])
def test_a_prompt_given_as_several_entries_on_one_row(cuts, dim):
    """Entries that end on an even slot and begin on the odd one behind it write halves of the same bytes in one call."""
    T, heads = 64, 2
    rng = np.random.default_rng(dim)
    k, v = (torch.from_numpy(rng.standard_normal((T, heads, dim)).astype(np.float32)).cuda().to(torch.bfloat16) for _ in range(2))
    ends = [0] + cuts + [T]
    cache = _fresh(dim=dim)
    table = torch.tensor([[2, 0, 3, 1]] * (len(ends) - 1), dtype=torch.int32, device="cuda")
    lens = torch.tensor(ends[:-1], dtype=torch.int32, device="cuda")
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_append(cache, k, v, table, lens, cu)
    got_k, got_v = _raw(cache)
    for got, want in ((got_k, k), (got_v, v)):
        rows = np.concatenate([got[p].swapaxes(0, 1) for p in (2, 0, 3, 1)])
        assert np.array_equal(rows, ref.rounded(want.double().cpu().numpy()))


@pytest.mark.parametrize("at", [0, 1, 6, 7, 14, 15])
def test_writing_one_slot_again_leaves_the_others(at):
    f = Filled([16], 2, 128, 16)
    new = torch.randn(2, 1, 2, 128, device="cuda").to(torch.bfloat16)
    block_ops.wd_kv4_append(f.cache, new[0], new[1], f.table_d, torch.tensor([at], dtype=torch.int32, device="cuda"))
    page = int(f.table_d[0, 0])
    for got, held, one in zip(_raw(f.cache), (f.k64, f.v64), new):
        held[at] = ref.rounded(one[0].double().cpu().numpy())
        assert np.array_equal(got[page].swapaxes(0, 1), held)
