"""The operators together: decode steps of a whole layer.

Each stage is compared with its definition in 64 bits on the inputs that it had
(the layer keeps its buffers), with the operators' own tolerances; the MoE part bit for
bit with a call of its own.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops, ops, workload
from output_centric_expert_gb300.decoder_layer import DecoderLayer, LayerWeights

from . import _block_ref as ref

pytestmark = pytest.mark.gpu


def _n(t):
    return t.double().cpu().numpy()


@pytest.fixture(scope="module")
def layer():
    s = workload.SHAPES["tiny"]
    torch.manual_seed(3)
    q_heads, kv_heads, dim = 4, 2, 64

    def norm():
        return 1 + 0.1 * torch.randn(s.H, device="cuda")
    qkv = torch.randn((q_heads + 2 * kv_heads) * dim, s.H, device="cuda") * 0.1
    o = torch.randn(s.H, q_heads * dim, device="cuda") * 0.1
    g, u, d = workload.all_weights(s, seed=0)
    moe = ops.DeviceWeights(ops.make_shape(s.H, s.I, s.E, s.top_k),
                            ops.moe_pack_weights(ops.make_shape(s.H, s.I, s.E, s.top_k), g, u, d))
    w = LayerWeights(block_ops.Fp4Weights.quantize(qkv), block_ops.Fp4Weights.quantize(o),
                     torch.randn(s.E, s.H, device="cuda"), moe, norm(), norm(), norm(), norm(),
                     torch.rand(1, s.H, device="cuda"))
    layer = DecoderLayer(w, block_ops.Kv4Cache(40, 16, kv_heads, dim), q_heads, max_batch=20, max_positions=64)
    layer.qkv64, layer.o64 = ref.rounded(_n(qkv)), ref.rounded(_n(o))
    return layer


def _close_matvec(y, x, w, rel):
    K = w.shape[1]
    mag = np.abs(_n(x)) @ np.abs(w).T
    want = _n(x) @ w.T
    tol = (K / 16 + 32) * 2.0 ** -23 * mag + 2.0 ** -40 * np.abs(_n(x)).max(1)[:, None] * np.abs(w).sum(1) + rel * np.abs(want)
    assert (np.abs(_n(y) - want) <= tol + 2.0 ** -120).all()


@pytest.mark.parametrize("B", [1, 3, 20])
def test_steps(layer, B):
    w, c = layer.w, layer.cache
    rng = np.random.default_rng(B)
    table = torch.from_numpy(rng.permutation(40)[:2 * B].reshape(B, 2).astype(np.int32)).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    keys = [[] for _ in range(B)]
    for _ in range(18):  # past a page
        res = torch.randn(B, layer.w.moe.shape.H, device="cuda").to(torch.bfloat16)
        before = res.clone()
        assert layer.step(res, table, lens, err) is res
        lens += 1
        for i in range(B):
            keys[i].append(_n(layer.qkv[i].view(-1, c.dim)[layer.q_heads:]))
    assert int(err) == 0
    # the last step, stage by stage
    a = _n(layer.a[:B])
    want = ref.norm(_n(before), None, None, None, _n(w.attn_pre), 1.0, float(np.float32(1e-6)))[1]
    assert (np.abs(a - want) <= 2.0 ** -8 * 1.02 * np.abs(want) + 2.0 ** -20).all()
    # v is as the projection gave it (q and k were rotated in place)
    v0 = (layer.q_heads + c.heads) * c.dim
    _close_matvec(layer.qkv[:B, v0:], layer.a[:B], layer.qkv64[v0:], 2.0 ** -8 * 1.01)
    for i in range(B):
        got = _n(layer.qkv[i].view(-1, c.dim)[:layer.q_heads + c.heads])
        plain = _n(layer.a[i]) @ layer.qkv64[:v0].T
        lo, hi = np.split(plain.reshape(-1, c.dim), 2, -1)
        angle = 17 * 10000.0 ** (-np.arange(0, c.dim, 2) / c.dim)
        want = np.concatenate([lo * np.cos(angle) - hi * np.sin(angle), hi * np.cos(angle) + lo * np.sin(angle)], -1)
        size = np.hypot(lo, hi)
        assert (np.abs(got - want) <= 2.0 ** -6 * np.concatenate([size, size], -1) + 1e-3).all()
        kv = ref.rounded(np.stack(keys[i]))  # [18, 2 * kv_heads, dim]
        q = _n(layer.qkv[i].view(-1, c.dim)[:layer.q_heads])
        out, _, mag, reach = ref.attend(q, kv[:, :c.heads], kv[:, c.heads:], c.dim ** -0.5)
        d = ((c.dim / 32 + 32) * 2.0 ** -23 + 2.0 ** -22) * reach[:, None]
        tol = (2 * d + 2.0 ** -11 + 2.0 ** -19) * mag + (18 * 2.0 ** -30 + 2.0 ** -22) * np.abs(kv).max() + 2.0 ** -8 * 1.01 * np.abs(out)
        assert (np.abs(_n(layer.attn[i]) - out) <= tol + 2.0 ** -25).all()
    _close_matvec(layer.o[:B], layer.attn[:B].view(B, -1), layer.o64, 2.0 ** -24)
    eps = float(np.float32(1e-6))
    r, m, mag = ref.norm(_n(before), _n(layer.o[:B]), _n(w.attn_post), None, _n(w.moe_pre), 1.0, eps)
    inv = np.abs(_n(w.moe_pre)) / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    assert (np.abs(_n(layer.m[:B]) - m) <= 2.0 ** -18 * mag * inv + 2.0 ** -8 * 1.02 * np.abs(m) + 2.0 ** -20).all()
    ids, wts = torch.empty_like(layer.ids[:B]), torch.empty_like(layer.wts[:B])
    ops.moe_route(w.moe.shape, torch.mm(layer.m[:B].float(), w.router.T), ids, wts)
    y = ops.moe_layer(w.moe, layer.m[:B], ids, wts, torch.empty_like(layer.h[:B]), torch.empty_like(layer.y[:B]))
    assert torch.equal(y, layer.y[:B]) and torch.equal(ids, layer.ids[:B])
    r1 = torch.from_numpy(r).to(torch.bfloat16).double().numpy()  # the residual between the blocks is kept in BF16
    r2, _, mag = ref.norm(r1, _n(layer.y[:B]), _n(w.moe_post), _n(w.moe_gate), None, 1.0, eps)
    # (a rounding of r1 may fall the other way)
    assert (np.abs(_n(res) - r2) <= 2.0 ** -7 * np.abs(r1) + 2.0 ** -18 * mag + 2.0 ** -8 * 1.01 * np.abs(r2) + 2.0 ** -25).all()


def test_refuses_weights_of_another_shape(layer):
    with pytest.raises(ValueError, match="qkv"):
        DecoderLayer(layer.w, layer.cache, 2, max_batch=2, max_positions=8)
