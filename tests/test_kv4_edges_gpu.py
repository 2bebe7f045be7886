"""The 4-bit KV cache at the ends of its arguments' ranges."""
import pytest
import torch

from .test_kv4_gpu import Filled, _attend, _q

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
