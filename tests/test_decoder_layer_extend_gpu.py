"""A decoder layer with a rope: chunks of new tokens and steps, stage by stage against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops
from output_centric_expert_gb300.decoder_layer import DecoderLayer

from . import _block_ref as ref
from .test_decoder_layer_gpu import _close_matvec, _n, layer as plain_layer  # noqa: F401
from .test_rope_gpu import turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer(plain_layer):  # noqa: F811
    freqs = block_ops.rope_freqs(32, scaling="linear", factor=2.0)
    made = DecoderLayer(plain_layer.w, block_ops.Kv4Cache(40, 16, 2, 64), plain_layer.q_heads, max_batch=60, max_positions=None,
                        rope=block_ops.Rope(freqs, interleaved=True))
    made.freqs, made.qkv64, made.o64 = freqs.numpy(), plain_layer.qkv64, plain_layer.o64
    return made


def _stages(layer, before, res, pos, keys):
    """The stages of the last call up to the second norm. keys: per row, the sequence's K and V up to it."""
    w, T, D, n, kv = layer.w, res.shape[0], layer.cache.dim, layer.q_heads, layer.cache.heads
    qkv = _n(layer.qkv[:T]).reshape(T, -1, D)
    _close_matvec(layer.qkv[:T, n * D:], layer.a[:T], layer.qkv64[n * D:], 2.0 ** -8 * 1.01)  # k and v, as the projection gave them
    plain = (_n(layer.a[:T]) @ layer.qkv64[:n * D].T).reshape(T, n, D)
    want, size = turned(plain, pos, layer.freqs, True)
    assert (np.abs(qkv[:, :n] - want) <= 2.0 ** -6 * size + 2.0 ** -7 * np.abs(want) + 1e-3).all()
    for i in range(T):
        k, v = keys[i]
        out, _, mag, reach = ref.attend(qkv[i, :n], k, v, D ** -0.5)
        d = ((D / 16 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach[:, None]
        tol = (2 * d + 2.0 ** -11 + 2.0 ** -18) * mag + len(k) * 2.0 ** -30 * np.abs(v).max() + 2.0 ** -8 * 1.01 * np.abs(out)
        assert (np.abs(_n(layer.attn[i]) - out) <= tol + 2.0 ** -25).all(), i
    _close_matvec(layer.o[:T], layer.attn[:T].view(T, -1), layer.o64, 2.0 ** -24)
    eps = float(np.float32(1e-6))
    r, m, mag = ref.norm(_n(before), _n(layer.o[:T]), _n(w.attn_post), None, _n(w.moe_pre), 1.0, eps)
    inv = np.abs(_n(w.moe_pre)) / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    assert (np.abs(_n(layer.m[:T]) - m) <= 2.0 ** -18 * mag * inv + 2.0 ** -8 * 1.02 * np.abs(m) + 2.0 ** -20).all()
    assert torch.isfinite(res.float()).all()


def _kv(layer, T, pos):
    """The rows' K and V as the cache has to hold them, from the layer's buffer."""
    D, n, kv = layer.cache.dim, layer.q_heads, layer.cache.heads
    qkv = _n(layer.qkv[:T]).reshape(T, -1, D)
    return ref.rounded(turned(qkv[:, n:n + kv], pos, layer.freqs, True)[0]), ref.rounded(qkv[:, n + kv:])


def test_prompts_chunks_and_steps(layer):
    """Prompts of several lengths, a second chunk of two of them, and a step, over one cache."""
    rng = np.random.default_rng(1)
    table = torch.from_numpy(rng.permutation(40)[:16].reshape(4, 4).astype(np.int32)).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [(np.zeros((0, 2, 64)), np.zeros((0, 2, 64))) for _ in range(4)]
    torch.manual_seed(5)
    for news in ([17, 1, 30, 0], [8, 0, 3, 40], None):
        lens = [len(k) for k, _ in held]
        one = news is None
        news = [1] * 4 if one else news
        cu = np.concatenate([[0], np.cumsum(news)])
        T = int(cu[-1])
        res = torch.randn(T, layer.w.moe.shape.H, device="cuda").to(torch.bfloat16)
        before = res.clone()
        start = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if one:
            assert layer.step(res, table, start, err) is res
        else:
            assert layer.extend(res, table, start, torch.tensor(cu, dtype=torch.int32, device="cuda"), err) is res
        assert int(err) == 0
        pos = np.concatenate([np.arange(b, b + n) for b, n in zip(lens, news)])
        k, v = _kv(layer, T, pos)
        held = [tuple(np.concatenate([h, x[cu[s]:cu[s + 1]]]) for h, x in zip(held[s], (k, v))) for s in range(4)]
        keys = [tuple(x[:lens[s] + i + 1] for x in held[s]) for s in range(4) for i in range(news[s])]
        _stages(layer, before, res, pos, keys)
    # and the cache holds just that
    total = [len(k) for k, _ in held]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(total)]), dtype=torch.int32, device="cuda")
    got = [torch.empty(sum(total), 2, 64, device="cuda") for _ in range(2)]
    block_ops.wd_kv4_gather(layer.cache, table, torch.zeros(4, dtype=torch.int32, device="cuda"), *got, cu)
    for i in range(2):
        assert np.array_equal(_n(got[i]), np.concatenate([h[i] for h in held]))


def test_padding_rows_touch_nothing(layer):
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    start, cu = torch.tensor([3, 0], dtype=torch.int32, device="cuda"), torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    torch.manual_seed(0)
    x = torch.randn(20, layer.w.moe.shape.H, device="cuda").to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(rows):
        for t in layer.cache.tensors:
            t.zero_()
        return layer.extend(rows.clone(), table, start, cu, err), [t.clone() for t in layer.cache.tensors]
    (a, held), (b, held2) = run(x), run(torch.cat([x[:12], -x[12:]]))
    assert int(err) == 0 and torch.equal(a[:12], b[:12]) and all(torch.equal(s, t) for s, t in zip(held, held2))
    assert torch.isfinite(a.float()).all()


def test_refusals(layer, plain_layer):  # noqa: F811
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    args = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), cu
    with pytest.raises(ValueError, match="rope"):
        plain_layer.extend(torch.zeros(1, layer.w.moe.shape.H, device="cuda"), *args)
    with pytest.raises(ValueError, match="61 tokens"):
        layer.extend(torch.zeros(61, layer.w.moe.shape.H, device="cuda"), *args)
    with pytest.raises(ValueError, match="rope"):
        DecoderLayer(layer.w, layer.cache, layer.q_heads, 2, None, rope=block_ops.Rope(block_ops.rope_freqs(128)))
    with pytest.raises(ValueError, match="max_positions"):
        DecoderLayer(layer.w, layer.cache, layer.q_heads, 2, None)
