"""Attention of several new tokens per sequence over the 4-bit cache, against its definition in 64 bits.

Tolerance, from the cached values: a logit's products are exact and summed in FP32, at most
D / 16 + 32 roundings or cuts in a row, so it is off by d = (D / 16 + 32) 2^-23 sum|q k| scale,
plus 2^-22 of itself for the scale factor; a probability by twice that, by 2^-19 for the
exponentials and joins, by 2^-11 (or 2^-30 of the largest value) where it is rounded to what
the tensor cores take; the sum over n keys by (n / 16 + 32) 2^-23 of the magnitudes. One
rounding to the output's type at the end.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref
from .test_kv4_gpu import ROUND, TYPES, Filled

pytestmark = pytest.mark.gpu


class Chunk(Filled):
    """A cache whose sequences end in new[s] new tokens each, and queries for these."""

    def __init__(self, before, new, heads, group, dim, page, kind="bf16", seed=0, edit=None, extra=0, pad=0, lead=0):
        super().__init__([a + b for a, b in zip(before, new)], heads, dim, page, kind, seed, edit=edit)
        self.before, self.new, self.kind, self.group = list(before), list(new), kind, group
        self.T = lead + sum(new) + extra
        wide = self.rng.standard_normal((self.T, heads * group + pad, dim)).astype(np.float32)
        self.q = torch.from_numpy(wide).to(TYPES[kind]).cuda()[:, :heads * group]
        self.start = torch.tensor(self.before, dtype=torch.int32, device="cuda")
        self.rows = np.concatenate([[0], np.cumsum(new)]) + lead
        self.cu_new = torch.tensor(self.rows, dtype=torch.int32, device="cuda")

    def run(self, window=0, scale=None, work=None, table=None, start=None, one_each=False, pad=0, **kw):
        T, H, D = self.q.shape
        out = torch.full((T, H + pad, D), 3.0, dtype=self.q.dtype, device="cuda")[:, :H]
        lse = torch.full((T, H), 3.0, device="cuda")
        work = block_ops.kv4_chunk_workspace(self.cache, T, H) if work is None else work
        got = block_ops.wd_kv4_attend_chunk(self.cache, self.q, self.table_d if table is None else table, self.start if start is None else start,
                                            out, work, None if one_each else self.cu_new, lse=lse, scale=scale, window=window, **kw)
        assert got is out
        return out, lse

    def check(self, out, lse, window=0, scale=None, seqs=None, rows=None):
        D, H = self.cache.dim, self.q.shape[1]
        scale = float(np.float32(D ** -0.5 if scale is None else scale))
        q, o, l = (t.double().cpu().numpy() for t in (self.q, out, lse))
        for s in range(len(self.new)) if seqs is None else seqs:
            k, v = self.of(s)
            b, n, r0 = self.before[s], self.new[s], int(self.rows[s])
            if not n:
                continue
            pos, key = np.arange(b, b + n)[:, None], np.arange(b + n)[None]
            seen = (key <= pos) & ((key > pos - window) if window else True)
            for h in range(H):
                kk, vv, qq = k[:, h // self.group], v[:, h // self.group], q[r0:r0 + n, h]
                z = np.where(seen, qq @ kk.T * scale, -np.inf)
                top = z.max(1, keepdims=True)
                p = np.exp(z - top)
                total = p.sum(1, keepdims=True)
                wl = (top + np.log(total))[:, 0]
                p /= total
                want, mag = p @ vv, p @ np.abs(vv)
                reach = np.where(seen, np.abs(qq) @ np.abs(kk).T, 0).max(1)[:, None] * abs(scale)
                d = ((D / 16 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach
                m = seen.sum(1)[:, None]
                tol = (2 * d + 2.0 ** -11 + 2.0 ** -19 + (m / 16 + 32) * 2.0 ** -23) * mag + m * 2.0 ** -30 * np.abs(vv).max() \
                    + ROUND[self.kind] * 1.01 * np.abs(want) + 2.0 ** -25
                off = np.abs(o[r0:r0 + n, h] - want)
                assert (off <= tol).all(), (s, h, (off / tol).max(), np.argwhere(off > tol)[:4])
                assert (np.abs(l[r0:r0 + n, h] - wl) <= d[:, 0] + 2.0 ** -19 + np.abs(wl) * 2.0 ** -22).all(), (s, h)


@pytest.mark.parametrize("before,new", [(0, 1), (0, 2), (1, 1), (15, 1), (15, 2), (16, 16), (0, 17), (127, 1), (127, 2), (128, 128), (100, 129),
                                        (0, 300), (255, 40), (1000, 5), (2049, 130)])
@pytest.mark.parametrize("dim,kind", [(64, "bf16"), (128, "bf16"), (128, "f16"), (256, "bf16"), (256, "f16")])
def test_lengths(before, new, dim, kind):
    c = Chunk([before], [new], 1, 3, dim, 16, kind, seed=new)
    c.check(*c.run())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 16, 17, 40, 130, 300])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 16), (256, 32)])
def test_head_layouts(group, dim, page, kind):
    c = Chunk([200, 0, 40, 0], [37, 0, 3, 50], 2 if group < 100 else 1, group, dim, page, kind, seed=group, pad=1)
    c.check(*c.run(pad=2))


@pytest.mark.parametrize("window", [1, 7, 16, 100, 128, 129, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows(window, dim):
    c = Chunk([300, 16, 1, 0, 999], [60, 1, 200, 5, 130], 1, 4, dim, 16, seed=window % 1000)
    c.check(*c.run(window=window), window=window)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_ragged_batches(page):
    """Many sequences and some that are far longer: rows whole in a CTA, rows cut over many."""
    rng = np.random.default_rng(page)
    before = [7000, 0] + [int(x) for x in rng.integers(0, 400, 30)] + [0, 0, 3000]
    new = [9, 700] + [int(x) for x in rng.integers(0, 12, 30)] + [1, 0, 150]
    c = Chunk(before, new, 3, 4, 64, page, seed=page)
    work = block_ops.kv4_chunk_workspace(c.cache, c.T, 12)
    first = c.run(work=work)
    c.check(*first)
    work.fill_(255)  # what the workspace holds does not matter
    again = c.run(work=work)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_one_token_each_is_the_decode_attention():
    """cu_new may be left out, and a single new token per sequence gives what wd_kv4_attend does, to rounding."""
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 300, 40)]
    c = Chunk(lens, [1] * 40, 2, 8, 128, 16)
    out, lse = c.run()
    c.check(out, lse)
    alone, lse1 = c.run(one_each=True)
    assert torch.equal(out, alone) and torch.equal(lse, lse1)
    step, lse2 = torch.empty_like(out), torch.empty_like(lse)
    block_ops.wd_kv4_attend(c.cache, c.q, c.table_d, c.start + 1, step, block_ops.kv4_workspace(c.cache, 40, 16), lse=lse2)
    assert ((out.float() - step.float()).abs() <= 2.0 ** -7 * step.float().abs() + 2.0 ** -9).all()
    assert ((lse - lse2).abs() <= 2.0 ** -16).all()


def test_more_sequences_than_threads():
    rng = np.random.default_rng(3)
    c = Chunk([int(x) for x in rng.integers(0, 40, 1500)], [int(x) for x in rng.integers(0, 4, 1500)], 1, 2, 64, 16)
    c.check(*c.run())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0, -0.3])
def test_scales(scale, kind):
    c = Chunk([300, 20], [100, 70], 2, 4, 128, 32, kind)
    c.check(*c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_values_of_very_different_sizes(kind):
    """V blocks whose scales differ by far more than f16 holds, in both orders of appearance, and zero blocks."""
    up = 2.0 ** (100 if kind == "bf16" else 10)
    down = 2.0 ** (-60 if kind == "bf16" else -14)

    def edit(k, v):
        n = v.shape[0]
        v[: n // 2, 0, :32] *= down
        v[n // 2:, 0, 32:64] *= down
        v[:, 0, 64:96] *= up
        v[:, 1, :32] = 0
        v[::3, 1, 96:] *= 2.0 ** -14
        k[:, 1] *= down
    c = Chunk([400], [200], 2, 2, 128, 16, kind, edit=edit)
    out, lse = c.run()
    k, v = c.of(0)
    seen = np.arange(600)[None] <= np.arange(400, 600)[:, None]
    for h in range(4):
        q = c.q[:, h].double().cpu().numpy()
        z = np.where(seen, q @ k[:, h // 2].T * 128 ** -0.5, -np.inf)
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        reach = (np.abs(q) @ np.abs(k[:, h // 2]).T).max(1)[:, None] * 128 ** -0.5
        want, mag = p @ v[:, h // 2], p @ np.abs(v[:, h // 2])
        got = out[:, h].double().cpu().numpy()
        # to the magnitudes alone: no key is lost beside a larger one
        tol = (2 * ((128 / 16 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach + 2.0 ** -11 + 2.0 ** -19 + 70 * 2.0 ** -23) * mag \
            + ROUND[kind] * 1.01 * np.abs(want) + (2.0 ** -133 if kind == "bf16" else 2.0 ** -25)
        assert (np.abs(got - want) <= tol).all(), h


def test_loud_queries():
    c = Chunk([150], [90], 1, 4, 128, 16)
    c.q[3, 0] *= 2.0 ** 100  # logits past what exp takes: one key wins
    c.q[:, 1] *= 2.0 ** -120
    c.q[5, 2, 5] = float("nan")
    c.q[:, 3] = 0
    out, lse = c.run()
    k, v = c.of(0)
    win = np.argmax(k[:154, 0] @ c.q[3, 0].double().cpu().numpy())
    assert np.array_equal(out[3, 0].double().cpu().numpy(), torch.from_numpy(v[win, 0]).to(torch.bfloat16).double().numpy())
    assert torch.isnan(out[5, 2]).all() and torch.isnan(lse[5, 2])
    assert torch.isfinite(out).all(-1).sum() == 90 * 4 - 1
    for i in (0, 89):
        mean = v[:151 + i].mean(0)[0]
        tol = 2.0 ** -8 * np.abs(mean) + 2.0 ** -11 * np.abs(v).mean()
        assert (np.abs(out[i, 3].double().cpu().numpy() - mean) <= tol).all()
        assert (np.abs(out[i, 1].double().cpu().numpy() - mean) <= tol).all()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 2), (128, 5), (256, 3)])
def test_nan_blocks_poison_only_rows_that_see_them(dim, group, window):
    """A NaN block of a value, and of a key, in tiles that rows see, and in those that only later rows or no row do."""
    def edit(k, v):
        v[37, 0, 40] = np.nan
        v[190, 0, 3] = np.inf
        v[205, 1, 50] = np.nan
        k[195, 1, 3] = np.nan

    args = [150, 30], [100, 5], 2, group, dim, 16
    c, clean = Chunk(*args, edit=edit), Chunk(*args)
    (out, lse), (good, glse) = c.run(window=window), clean.run(window=window)
    pos = torch.arange(150, 250, device="cuda")

    def sees(key):
        return (pos >= key) & (pos < key + window if window else pos >= 0)
    bad = torch.zeros(105, 2 * group, dim, dtype=torch.bool, device="cuda")
    bad[:100, :group, 32:64] |= sees(37)[:, None, None]
    bad[:100, :group, :32] |= sees(190)[:, None, None]
    bad[:100, group:, 32:64] |= sees(205)[:, None, None]
    bad[:100, group:] |= sees(195)[:, None, None]
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], good[~bad])
    assert torch.equal(torch.isnan(lse[:100, group:]), sees(195)[:, None].expand(100, group))
    assert torch.equal(lse[:, :group], glse[:, :group])


def test_what_has_no_page_is_flagged_and_left_out():
    c = Chunk([64, 40], [20, 9], 1, 2, 64, 16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.run(err_flag=err)
    assert int(err) == 0
    table = c.table.copy()
    table[0, 1], table[0, 3] = -1, c.cache.pages
    out, lse = c.run(table=torch.from_numpy(table).cuda(), err_flag=err)
    assert int(err) == 1
    k, v = c.of(0)
    keep = np.r_[0:16, 32:48, 64:84]
    g = Chunk([32], [20], 1, 2, 64, 16)
    g.k64, g.v64, g.q = k[keep], v[keep], c.q[:20]
    g.check(out[:20], lse[:20])
    c.check(out, lse, seqs=[1])
    # no page at all; and a negative length
    err.zero_()
    table = c.table.copy()
    table[0] = -1
    out, lse = c.run(table=torch.from_numpy(table).cuda(), start=torch.tensor([64, -2], dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err) == 1 and (out == 0).all() and (lse == -float("inf")).all()
    # positions past the table's row: its keys count
    err.zero_()
    out, lse = c.run(start=torch.tensor([1 << 30, 40], dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err) == 1
    c.check(out, lse, seqs=[1])
    assert c.table.shape[1] == 6
    err.zero_()
    out, lse = c.run(start=torch.tensor([96, 40], dtype=torch.int32, device="cuda"), window=20, err_flag=err)  # the last rows see nothing
    assert int(err) == 1 and (out[19] == 0).all() and torch.isinf(lse[19]).all()


def test_rows_of_no_sequence_stay_as_they_are():
    c = Chunk([30, 0, 8], [70, 0, 13], 2, 3, 128, 16, extra=50, lead=7, pad=2)
    out, lse = c.run(pad=1)
    c.check(out, lse)
    for t in (out, lse):
        assert (t[:7] == 3).all() and (t[90:] == 3).all()


@pytest.mark.parametrize("dim,group,new", [(64, 1, 1), (64, 3, 5), (128, 1, 2), (128, 12, 30), (256, 9, 3), (128, 8, 16)])
@pytest.mark.parametrize("before", [[40001], [20000, 5, 7777, 0, 300]])
def test_rows_of_many_parts(before, dim, group, new):
    c = Chunk(before, [new] * len(before), 1, group, dim, 32, seed=group)
    out, lse = c.run()
    c.check(out, lse)
    again, lse2 = c.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_a_long_prompt(kind):
    c = Chunk([0], [2500], 1, 4, 128, 64, kind)
    c.check(*c.run())


def test_streams_graphs_and_shared_workspaces():
    """Two captured calls that share a workspace and run one after the other, replayed on another stream."""
    a, b = Chunk([5000, 3], [6, 70], 1, 8, 128, 64), Chunk([900], [200], 2, 3, 64, 16, seed=1)
    want = [x.run() for x in (a, b)]
    work = torch.empty(max(block_ops.kv4_chunk_workspace(x.cache, x.T, x.q.shape[1]).numel() for x in (a, b)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in (a, b):
        out, lse = torch.empty_like(x.q), torch.empty(x.q.shape[:2], device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            block_ops.wd_kv4_attend_chunk(x.cache, x.q, x.table_d, x.start, out, work, x.cu_new, lse=lse)
        graphs.append(g)
        got.append((out, lse))
    for _ in range(3):
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
    side.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))
    out = torch.empty_like(a.q)
    block_ops.wd_kv4_attend_chunk(a.cache, a.q, a.table_d, a.start, out, work, a.cu_new, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0][0])


def test_lengths_may_change_under_a_graph():
    c = Chunk([300, 100], [40, 40], 1, 4, 128, 16)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")
    work = block_ops.kv4_chunk_workspace(c.cache, c.T, 4)
    cu, start = c.cu_new.clone(), c.start.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block_ops.wd_kv4_attend_chunk(c.cache, c.q, c.table_d, start, out, work, cu, lse=lse)
    g.replay()
    c.check(out, lse)
    c.before, c.new = [320, 60], [20, 60]
    c.rows = np.array([0, 20, 80])
    start.copy_(torch.tensor(c.before))
    cu.copy_(torch.tensor(c.rows))
    c.of = lambda s: tuple(x[(0, 340)[s]:(340, 460)[s]] for x in (c.k64, c.v64))
    g.replay()
    c.check(out, lse)


def test_a_cache_past_four_gib():
    pages = (1 << 32) // (256 * 8 * 128) + 2
    cache = block_ops.Kv4Cache(pages, 256, 8, 256)
    k = torch.randn(20, 8, 256, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lens, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_append(cache, k, k.neg(), table, lens, cu)
    c = object.__new__(Chunk)
    c.cache, c.before, c.new, c.lens, c.kind, c.group, c.T = cache, [0], [20], [20], "bf16", 2, 20
    c.table_d, c.start, c.cu_new, c.rows = table, lens, cu, [0, 20]
    c.k64 = ref.rounded(k.double().cpu().numpy())
    c.v64 = -c.k64
    c.q = torch.randn(20, 16, 256, device="cuda").to(torch.bfloat16)
    c.check(*c.run())


def test_empty_calls_and_refusals():
    c = Chunk([5], [3], 2, 2, 64, 16)
    work = block_ops.kv4_chunk_workspace(c.cache, 3, 4)
    args = c.table_d, c.start
    none = c.q[:0].contiguous()
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_attend_chunk(c.cache, none, *args, none.clone(), work, zero)
    with pytest.raises(block_ops.WarpDecodeError, match="workspace"):
        block_ops.wd_kv4_attend_chunk(c.cache, c.q, *args, c.q.clone(), work[:8], c.cu_new)
    with pytest.raises(block_ops.WarpDecodeError) as e:
        block_ops.wd_kv4_attend_chunk(c.cache, c.q[:, :3].contiguous(), *args, c.q[:, :3].contiguous(), work, c.cu_new)
    assert e.value.status == 2
    with pytest.raises(block_ops.WarpDecodeError):  # three rows, one sequence
        block_ops.wd_kv4_attend_chunk(c.cache, c.q, *args, c.q.clone(), work)
    with pytest.raises(TypeError):
        block_ops.wd_kv4_attend_chunk(c.cache, c.q, *args, c.q.float(), work, c.cu_new)
    with pytest.raises(TypeError):
        block_ops.wd_kv4_attend_chunk(c.cache, c.q, *args, c.q.clone(), work, c.cu_new.long())
    with pytest.raises(ValueError):
        block_ops.kv4_chunk_workspace(c.cache, 3, 3)
