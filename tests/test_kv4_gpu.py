"""The 4-bit KV cache on the GPU: append, gather and attention against their definitions in 64 bits.

Tolerance of the attention, from the cached values: a logit's products are exact and
pass at most D/32 + 32 FP32 additions in a row, so it is off by d = (D/32 + 32) 2^-23
sum|q k| scale, plus 2^-22 of itself for the scale factor; a probability by twice
that, by 2^-20 for the exponentials and joins and by 2^-11 where it is rounded to
f16 (or by 2^-30 absolute, below f16's normal range); a key whose V scale is below
2^-23 of its block's largest may add nothing; the sum over keys by 2^-20 of the
magnitudes. One rounding to the output's type at the end.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


class Filled:
    """A cache with sequences of the given lengths on shuffled pages, and their values (numpy)."""

    def __init__(self, lens, heads, dim, page, kind="bf16", seed=0, spare=3, edit=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens = rng, list(lens)
        per = [-(-n // page) for n in lens]
        pages = rng.permutation(sum(per) + spare).astype(np.int32)
        self.table = np.full((len(lens), max(per + [1])), -1, np.int32)  # unused entries name no page
        for i, n in enumerate(per):
            self.table[i, :n] = pages[sum(per[:i]):sum(per[:i]) + n]
        self.cache = block_ops.Kv4Cache(sum(per) + spare, page, heads, dim)
        for t in self.cache.tensors:
            t.fill_(255)  # what nothing wrote: NaN scales
        T = sum(lens)
        k = (rng.standard_normal((T, heads, dim)) * (1 + 5 * (rng.random((1, heads, dim)) < 0.05))).astype(np.float32)
        v = rng.standard_normal((T, heads, dim)).astype(np.float32)
        if edit:
            edit(k, v)
        self.k, self.v = (torch.from_numpy(a).to(TYPES[kind]).cuda() for a in (k, v))
        self.table_d = torch.from_numpy(self.table).cuda()
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        block_ops.wd_kv4_append(self.cache, self.k, self.v, self.table_d, torch.zeros_like(self.lens_d), self.cu)
        self.k64, self.v64 = (ref.rounded(a.double().cpu().numpy()) for a in (self.k, self.v))

    def of(self, s):
        a = sum(self.lens[:s])
        return self.k64[a:a + self.lens[s]], self.v64[a:a + self.lens[s]]


def _raw(cache):
    """The cache's bytes as (k values, v values) [pages, heads, page, dim], read by the documented layout."""
    P, H, D, N = cache.page_size, cache.heads, cache.dim, cache.pages
    kc, ks, vc, vs = (t.cpu().numpy() for t in cache.tensors)
    kc = kc.reshape(N, H, P, 4, D // 32, 4)
    vc = vc.reshape(N, H, P // 2, 8, D // 32, 4)
    slot, d = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    kb = kc[:, :, slot, d % 32 // 8, d // 32, d % 8 // 2]
    vb = vc[:, :, slot // 2, d % 32 // 4, d // 32, d % 4]
    vs = vs.reshape(N, H, P // 2, D // 32, 2).swapaxes(3, 4).reshape(N, H, P, D // 32)
    return [ref.values((b >> (4 * (n % 2))) & 15, s) for b, n, s in ((kb, d, ks.reshape(N, H, P, D // 32)), (vb, slot, vs))]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lens,heads,dim,page", [
    ([1], 1, 64, 16), ([5, 0, 33, 16], 2, 128, 16), ([70, 1, 64], 3, 256, 32), ([300, 129], 1, 128, 128),
    ([257], 5, 64, 256), ([63, 65], 2, 128, 64), ([31, 18], 17, 64, 16), ([9, 40], 9, 256, 32)])
def test_append_writes_the_documented_layout(lens, heads, dim, page, kind):
    f = Filled(lens, heads, dim, page, kind)
    k, v = _raw(f.cache)
    written = np.zeros((f.cache.pages, page), bool)
    for s, n in enumerate(lens):
        ks, vs = f.of(s)
        for j in range(n):
            at = f.table[s, j // page], slice(None), j % page
            written[at[0], at[2]] = True
            assert np.array_equal(k[at], ks[j]) and np.array_equal(v[at], vs[j]), (s, j)
    assert np.isnan(k.swapaxes(1, 2)[~written]).all() and np.isnan(v.swapaxes(1, 2)[~written]).all()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 16), (256, 16)])
def test_gather_reads_back_and_steps_extend(dim, page, out):
    f = Filled([20, 0, 15, 47], 2, dim, page, spare=8)
    # one more token each, by a step without cu_new; pages for it from the spare ones
    used = set(f.table[f.table >= 0].tolist())
    free = [p for p in range(f.cache.pages) if p not in used]
    table = np.concatenate([f.table, np.full((4, 1), -1, np.int32)], 1)
    for s, n in enumerate(f.lens):
        if n % page == 0:
            table[s, n // page] = free.pop()
    table_d = torch.from_numpy(table).cuda()
    wide = torch.randn(4, 3 * 2 * dim, device="cuda").to(torch.bfloat16)  # q, k, v side by side
    k1, v1 = (wide[:, i * 2 * dim:(i + 1) * 2 * dim].view(4, 2, dim) for i in (1, 2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_append(f.cache, k1, v1, table_d, f.lens_d, err_flag=err)
    new = torch.tensor(np.concatenate([[0], np.cumsum(np.array(f.lens) + 1)]), dtype=torch.int32, device="cuda")
    T = int(new[-1])
    k, v = (torch.empty(T, 2, dim, dtype=TYPES[out], device="cuda") for _ in range(2))
    block_ops.wd_kv4_gather(f.cache, table_d, torch.zeros_like(f.lens_d), k, v, new, err)
    assert int(err) == 0
    k2, v2 = (ref.rounded(t.double().cpu().numpy()) for t in (k1, v1))
    for s in range(4):
        ks, vs = f.of(s)
        a, b = int(new[s]), int(new[s + 1])
        for got, old, one in ((k, ks, k2), (v, vs, v2)):
            want = np.concatenate([old, one[s:s + 1]])
            want = torch.from_numpy(want).to(TYPES[out]).double().numpy()
            assert np.array_equal(got[a:b].double().cpu().numpy(), want)


@pytest.mark.parametrize("steps", [[1] * 9, [3, 1, 4, 1], [1, 2, 2, 4], [2, 7]])
def test_steps_join_keys_that_share_bytes(steps):
    """Two neighbouring keys' V share bytes: appended together or one by one, they are the same."""
    rng = np.random.default_rng(len(steps))
    cache = block_ops.Kv4Cache(4, 16, 2, 128)
    for t in cache.tensors:
        t.fill_(255)
    k, v = (torch.from_numpy(rng.standard_normal((2, 9, 2, 128)).astype(np.float32)).cuda().to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[2], [1]], dtype=torch.int32, device="cuda")
    at = 0
    for n in steps:
        cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
        lens = torch.full((2,), at, dtype=torch.int32, device="cuda")
        block_ops.wd_kv4_append(cache, k[:, at:at + n].reshape(2 * n, 2, 128), v[:, at:at + n].reshape(2 * n, 2, 128), table, lens, cu)
        at += n
    got_k, got_v = _raw(cache)
    for s, page in enumerate((2, 1)):
        assert np.array_equal(got_k[page].swapaxes(0, 1)[:9], ref.rounded(k[s].double().cpu().numpy()))
        assert np.array_equal(got_v[page].swapaxes(0, 1)[:9], ref.rounded(v[s].double().cpu().numpy()))


def test_special_blocks():
    def edit(k, v):
        k[0, 0, :32], v[0, 0, 32:64] = 0, 0
        k[1, 0, 3], v[1, 0, 40], k[2, 1, 70] = np.inf, np.nan, -np.inf
        k[3] *= 1e-30
        v[3] *= 1e30
        k[4, 0, :4] = [7.9, 5, 2.5, 0.25]
    f = Filled([9], 2, 128, 16, edit=edit)
    k, v = (torch.empty(9, 2, 128, dtype=torch.float32, device="cuda") for _ in range(2))
    block_ops.wd_kv4_gather(f.cache, f.table_d, torch.zeros_like(f.lens_d), k, v, f.cu)
    assert np.array_equal(k.double().cpu().numpy(), f.k64, equal_nan=True)
    assert np.array_equal(v.double().cpu().numpy(), f.v64, equal_nan=True)
    assert np.isnan(f.k64[1, 0, :32]).all() and np.isfinite(f.k64[1, 0, 32:]).all()


def test_tokens_that_have_no_place_are_flagged_and_left_out():
    cache = block_ops.Kv4Cache(4, 16, 1, 64)
    for t in cache.tensors:
        t.fill_(255)
    before = [t.clone() for t in cache.tensors]
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, -1], [1, 4], [2, 1 << 30], [3, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([16, 16, 16, 32], dtype=torch.int32, device="cuda")  # the last is beyond its row
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_append(cache, k, k, table, lens, err_flag=err)
    assert int(err) == 1 and all(torch.equal(a, b) for a, b in zip(cache.tensors, before))
    err.zero_()
    block_ops.wd_kv4_append(cache, k, k, table, torch.full_like(lens, -1), err_flag=err)
    assert int(err) == 1 and all(torch.equal(a, b) for a, b in zip(cache.tensors, before))
    # rows behind cu_new[S] are ignored without a flag
    err.zero_()
    cu = torch.tensor([0, 1, 1, 2, 2], dtype=torch.int32, device="cuda")
    out = torch.full((4, 1, 64), 5.0, device="cuda")
    block_ops.wd_kv4_append(cache, k, k, table, torch.zeros_like(lens), cu, err)
    block_ops.wd_kv4_gather(cache, table, torch.zeros_like(lens), out, out.clone(), cu, err)
    assert int(err) == 0 and (out[:2] == 1).all() and (out[2:] == 5).all()
    k, _ = _raw(cache)
    assert [np.isfinite(k[p]).any() for p in range(4)] == [True, False, True, False]


# ------------------------------------------------------------------ attention --

def _attend(f, q, window=0, scale=None, lens=None, table=None, work=None, **kw):
    S, H, D = q.shape
    out = torch.full_like(q, 3.0)
    lse = torch.full((S, H), 3.0, device="cuda")
    work = block_ops.kv4_workspace(f.cache, S, H) if work is None else work
    block_ops.wd_kv4_attend(f.cache, q, f.table_d if table is None else table, f.lens_d if lens is None else lens, out,
                            work, lse=lse, scale=scale, window=window, **kw)
    return out, lse


def _check(f, q, out, lse, window=0, scale=None, kind="bf16", lens=None):
    D = q.shape[2]
    scale = float(np.float32(D ** -0.5 if scale is None else scale))
    for s in range(q.shape[0]):
        k, v = f.of(s)
        n = f.lens[s] if lens is None else lens[s]
        lo = max(0, n - window) if window else 0
        k, v = k[lo:n], v[lo:n]
        want, wl, mag, reach = ref.attend(q[s].double().cpu().numpy(), k, v, scale)
        got, gl = out[s].double().cpu().numpy(), lse[s].double().cpu().numpy()
        if n - lo == 0:
            assert (got == 0).all() and (gl == -np.inf).all()
            continue
        d = ((D / 32 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach[:, None]
        most = np.abs(v).max()
        tol = (2 * d + 2.0 ** -11 + 2.0 ** -19) * mag + (n * 2.0 ** -30 + 2.0 ** -22) * most \
            + ROUND[kind] * 1.01 * np.abs(want) + 2.0 ** -25
        off = np.abs(got - want)
        assert (off <= tol).all(), (s, (off / tol).max())
        assert (np.abs(gl - wl) <= d[:, 0] + 2.0 ** -19 + np.abs(wl) * 2.0 ** -22).all(), (s, np.abs(gl - wl).max())


def _q(rng, S, H, D, kind="bf16", pad=0):
    wide = torch.from_numpy(rng.standard_normal((S, H + pad, D)).astype(np.float32)).to(TYPES[kind]).cuda()
    return wide[:, :H]


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257, 1000, 2049])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_lengths(n, dim):
    f = Filled([n], 2, dim, 16, seed=n)
    q = _q(f.rng, 1, 8, dim)
    _check(f, q, *_attend(f, q))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [1, 3, 5, 8, 9, 12, 16, 17, 40])
@pytest.mark.parametrize("dim,page", [(64, 64), (128, 16), (256, 32)])
def test_head_layouts(group, dim, page, kind):
    f = Filled([300, 0, 77], 2, dim, page, kind, seed=group)
    q = _q(f.rng, 3, 2 * group, dim, kind, pad=1)
    _check(f, q, *_attend(f, q), kind=kind)


@pytest.mark.parametrize("window", [1, 7, 16, 100, 255, 256, 5000])
def test_windows(window):
    f = Filled([300, 16, 1, 0, 999], 1, 128, 16, seed=window)
    q = _q(f.rng, 5, 4, 128)
    _check(f, q, *_attend(f, q, window=window), window=window)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_ragged_batches_share_rows_between_ctas(page):
    """Many sequences and one that is far longer: rows whole in a CTA, rows cut over many."""
    lens = [7000] + [int(x) for x in np.random.default_rng(page).integers(0, 400, 30)] + [0, 0, 3000]
    f = Filled(lens, 3, 64, page, seed=page)
    q = _q(f.rng, len(lens), 6, 64)
    work = block_ops.kv4_workspace(f.cache, len(lens), 6)
    first = _attend(f, q, work=work)
    _check(f, q, *first)
    work.fill_(255)  # what the workspace holds does not matter
    again = _attend(f, q, work=work)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    half = torch.tensor([n // 2 for n in lens], dtype=torch.int32, device="cuda")
    _check(f, q, *_attend(f, q, lens=half, work=work), lens=[n // 2 for n in lens])


def test_more_sequences_than_threads():
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 40, 700)]
    f = Filled(lens, 1, 64, 16)
    q = _q(f.rng, 700, 2, 64)
    _check(f, q, *_attend(f, q))


@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0, -0.3])
def test_scales(scale):
    f = Filled([400, 90], 2, 128, 32)
    q = _q(f.rng, 2, 8, 128)
    _check(f, q, *_attend(f, q, scale=scale), scale=scale)


def test_values_of_very_different_sizes():
    """V blocks whose scales differ by far more than f16 holds, in both orders of appearance, and zero blocks."""
    def edit(k, v):
        n = v.shape[0]
        v[: n // 2, 0, :32] *= 2.0 ** -60
        v[n // 2:, 0, 32:64] *= 2.0 ** -60
        v[:, 0, 64:96] *= 2.0 ** 100
        v[:, 1, :32] = 0
        v[::3, 1, 96:] *= 2.0 ** -18
        k[:, 1] *= 2.0 ** -100
    f = Filled([600], 2, 128, 16, edit=edit)
    q = _q(f.rng, 1, 4, 128)
    out, lse = _attend(f, q)
    want, wl, mag, reach = ref.attend(q[0].double().cpu().numpy(), *f.of(0), 128 ** -0.5)
    off = np.abs(out[0].double().cpu().numpy() - want).reshape(4, 4, 32)
    k, v = f.of(0)
    d = ((128 / 32 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach
    for h in range(4):
        for b in range(4):
            most = np.abs(v[:, h // 2, 32 * b:32 * b + 32]).max()
            tol = (2 * d[h] + 2.0 ** -11 + 2.0 ** -19) * mag[h, 32 * b:32 * b + 32] \
                + (600 * 2.0 ** -30 + 2.0 ** -22) * most + 2.0 ** -8 * 1.01 * np.abs(want[h, 32 * b:32 * b + 32])
            assert (off[h, b] <= tol + 2.0 ** -133).all(), (h, b)


def test_loud_queries_and_infinities():
    f = Filled([200, 50], 1, 128, 16)
    q = _q(f.rng, 2, 4, 128).clone()
    q[0, 0] *= 2.0 ** 100  # logits past what exp takes: one key wins
    q[0, 1] *= 2.0 ** -120
    q[1, 2, 5] = float("nan")
    q[1, 3] = 0
    out, lse = _attend(f, q)
    k, v = f.of(0)
    win = np.argmax(k[:, 0] @ q[0, 0].double().cpu().numpy())
    assert np.array_equal(out[0, 0].double().cpu().numpy(), torch.from_numpy(v[win, 0]).to(torch.bfloat16).double().numpy())
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    _check(f, q[:1, 1:], out[:1, 1:], lse[:1, 1:])
    got, want = out[1, 3].double().cpu().numpy(), f.of(1)[1].mean(0)[0]
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -11


def test_nan_blocks_poison_only_what_reads_them():
    def edit(k, v):
        v[37, 0, 40] = np.nan  # block 1 of one value
        k[250, 1, 3] = np.inf  # a key of head 1
    f = Filled([400, 30], 2, 128, 16, edit=edit)
    f2 = Filled([400, 30], 2, 128, 16)
    q = _q(f.rng, 2, 4, 128)
    (out, lse), (clean, _) = _attend(f, q), _attend(f2, q)
    assert torch.isnan(out[0, :2, 32:64]).all() and torch.isnan(out[0, 2:]).all()
    rest = [slice(0, 32), slice(64, 128)]
    assert all(torch.equal(out[0, :2, r], clean[0, :2, r]) for r in rest) and torch.equal(out[1], clean[1])
    short = torch.tensor([37, 30], dtype=torch.int32, device="cuda")  # the same pages, the NaN behind the end
    out, _ = _attend(f, q, lens=short)
    assert torch.isfinite(out).all()
    out, _ = _attend(f, q[:, :2].repeat(1, 2, 1)[:, :4], window=100)  # before the window
    assert torch.isfinite(out[0, :2]).all()


def test_what_has_no_page_is_flagged_and_left_out():
    f = Filled([64, 40], 1, 64, 16)
    q = _q(f.rng, 2, 2, 64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _attend(f, q, err_flag=err)
    assert int(err) == 0
    table = f.table.copy()
    table[0, 1], table[0, 3] = -1, f.cache.pages
    out, lse = _attend(f, q, table=torch.from_numpy(table).cuda(), err_flag=err)
    assert int(err) == 1
    k, v = f.of(0)
    keep = np.r_[0:16, 32:48]
    g = Filled([32], 1, 64, 16)
    g.k64, g.v64 = k[keep], v[keep]
    _check(g, q[:1], out[:1], lse[:1])
    err.zero_()  # longer than the table's row: the row's keys count; a negative length has none
    out, lse = _attend(f, q, lens=torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err) == 1
    _check(f, q[:1], out[:1], lse[:1])
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 3), (64, 16), (128, 1), (128, 12), (256, 1), (256, 9)])
@pytest.mark.parametrize("lens", [[40001], [20000, 5, 7777, 0, 300]])
def test_rows_of_many_parts(lens, dim, group):
    """Rows that many CTAs share, more of them than there are groups of sums to join for few heads."""
    f = Filled(lens, 1, dim, 32, seed=group)
    q = _q(f.rng, len(lens), group, dim)
    out, lse = _attend(f, q)
    _check(f, q, out, lse)
    again, lse2 = _attend(f, q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_long_sequence_and_another_stream():
    f = Filled([40001], 1, 128, 64)
    q = _q(f.rng, 1, 8, 128)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    work = block_ops.kv4_workspace(f.cache, 1, 8)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out, lse = _attend(f, q, work=work)
    side.synchronize()
    _check(f, q, out, lse)


def test_a_cache_past_four_gib():
    """Pages beyond 2^32 bytes of codes are addressed."""
    pages = (1 << 32) // (256 * 8 * 128) + 2
    cache = block_ops.Kv4Cache(pages, 256, 8, 256)
    k = torch.randn(20, 8, 256, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    block_ops.wd_kv4_append(cache, k, k.neg(), table, torch.zeros_like(lens), cu)
    assert int(cache.tensors[0][: 1 << 32].max()) == 0
    f = object.__new__(Filled)
    f.cache, f.lens, f.table_d, f.lens_d = cache, [20], table, lens
    f.k64 = ref.rounded(k.double().cpu().numpy())
    f.v64 = -f.k64
    q = torch.randn(1, 8, 256, device="cuda").to(torch.bfloat16)
    _check(f, q, *_attend(f, q))


def test_empty_calls_and_refusals():
    f = Filled([5], 2, 64, 16)
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    work = block_ops.kv4_workspace(f.cache, 1, 4)
    no_table, no_lens = f.table_d[:0], f.lens_d[:0]
    block_ops.wd_kv4_attend(f.cache, none, no_table, no_lens, none.clone(), work)
    block_ops.wd_kv4_append(f.cache, none[:, :2].contiguous(), none[:, :2].contiguous(), no_table, no_lens)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(block_ops.WarpDecodeError, match="workspace"):
        block_ops.wd_kv4_attend(f.cache, q, f.table_d, f.lens_d, q.clone(), work[:64])
    with pytest.raises(block_ops.WarpDecodeError) as e:
        block_ops.wd_kv4_attend(f.cache, q[:, :3].contiguous(), f.table_d, f.lens_d, q[:, :3].contiguous(), work)
    assert e.value.status == 2
    with pytest.raises(TypeError):
        block_ops.wd_kv4_attend(f.cache, q, f.table_d, f.lens_d, q.float(), work)
    with pytest.raises(TypeError):
        block_ops.wd_kv4_attend(f.cache, q, f.table_d.long(), f.lens_d, q.clone(), work)
    with pytest.raises(ValueError):
        block_ops.Kv4Cache(4, 24, 2, 64)
