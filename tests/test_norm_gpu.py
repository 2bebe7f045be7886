"""wd_block_norm against its formula in 64 bits.

Tolerances: the two sums of squares pass at most H/32 + 16 FP32 additions of
positive terms in a row, so the norms' factors are off by at most half of
(H/32 + 16) 2^-24 plus a few roundings; r' is off by that times |gate n| plus 2^-22
of what it sums; out by r's error times its factor and its own factor's.
"""
import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from . import _block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _t(a, kind):
    return torch.from_numpy(np.asarray(a, np.float32)).to(TYPES[kind]).cuda()


def _n(t):
    return None if t is None else t.double().cpu().numpy()


def _check(H, res, y, w_post, gate, w_pre, scale, eps, r_got, o_got, rk, ok):
    r, out, mag = ref.norm(_n(res), _n(y), _n(w_post), _n(gate), _n(w_pre), scale, eps)
    f = (H / 32 + 32) * 2.0 ** -24
    r_err = (f + 2.0 ** -22) * mag
    if r_got is not None:
        off = np.abs(_n(r_got) - r)
        assert (off <= r_err + ROUND[rk] * 1.01 * np.abs(r) + 2.0 ** -25).all(), off.max()
    if out is not None:
        inv = np.abs(_n(w_pre)) / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
        # an error in every r' moves the factor by at most their norms' ratio
        move = np.sqrt((r_err ** 2).mean(-1, keepdims=True) / ((r * r).mean(-1, keepdims=True) + eps))
        off = np.abs(_n(o_got) - out)
        assert (off <= r_err * inv + (f + move + 2.0 ** -21 + ROUND[ok] * 1.01) * np.abs(out) + 2.0 ** -25).all()


@pytest.mark.parametrize("H", [1, 7, 32, 64, 127, 512, 1000, 2048, 4096, 7167, 7168, 8191, 8192])
@pytest.mark.parametrize("T", [1, 3, 33])
@pytest.mark.parametrize("gate_kind", ["none", "channel", "token", "both", "one"])
def test_widths_and_gates(T, H, gate_kind):
    rng = np.random.default_rng(T * H)
    y, res = _t(rng.standard_normal((T, H)) * 3, "f32"), _t(rng.standard_normal((T, H)), "bf16")
    w_post, w_pre = _t(1 + rng.standard_normal(H) / 8, "f32"), _t(1 + rng.standard_normal(H) / 8, "f32")
    shape = {"none": None, "channel": (1, H), "token": (T, 1), "both": (T, H), "one": (1, 1)}[gate_kind]
    gate = None if shape is None else _t(rng.standard_normal(shape), "f32")
    r, o = torch.empty_like(res), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    block_ops.wd_block_norm(res, r, o, y=y, w_post=w_post, gate=gate, w_pre=w_pre, res_scale=0.7)
    _check(H, res, y, w_post, gate, w_pre, float(np.float32(0.7)), float(np.float32(1e-6)), r, o, "bf16", "bf16")


@pytest.mark.parametrize("T,H", [(3000, 255), (3000, 257), (5200, 511), (2600, 513), (2600, 1023), (1300, 1025), (700, 2049),
                                 (400, 4095), (200, 4097)])
@pytest.mark.parametrize("gate_kind", ["channel", "both"])
def test_odd_widths_of_many_rows(T, H, gate_kind):
    """Every number of threads that a row takes, and more rows than an SM has at a time."""
    rng = np.random.default_rng(T + H)
    y, res = _t(rng.standard_normal((T, H)) * 3, "f16"), _t(rng.standard_normal((T, H)), "f32")
    w_post, w_pre = _t(1 + rng.standard_normal(H) / 8, "bf16"), _t(1 + rng.standard_normal(H) / 8, "bf16")
    gate = _t(rng.standard_normal((1 if gate_kind == "channel" else T, H)), "bf16")
    r, o = torch.empty_like(res), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    block_ops.wd_block_norm(res, r, o, y=y, w_post=w_post, gate=gate, w_pre=w_pre, res_scale=0.7)
    _check(H, res, y, w_post, gate, w_pre, float(np.float32(0.7)), float(np.float32(1e-6)), r, o, "f32", "bf16")


@pytest.mark.parametrize("yk", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rk", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("wk,ok", [("f32", "bf16"), ("bf16", "f16"), ("f16", "f32")])
# 2048 and 3000: the ring of rows takes exactly the 48 KB that need no opt-in, beside the static memory
@pytest.mark.parametrize("H", [96, 2048, 2056, 3000])
def test_types(H, yk, rk, wk, ok):
    rng = np.random.default_rng(H)
    T = 5
    y, res = _t(rng.standard_normal((T, H)), yk), _t(rng.standard_normal((T, H)), rk)
    w_post, w_pre, gate = (_t(rng.standard_normal(s), wk) for s in ((H,), (H,), (T, H)))
    r, o = torch.empty_like(res), torch.empty(T, H, dtype=TYPES[ok], device="cuda")
    block_ops.wd_block_norm(res, r, o, y=y, w_post=w_post, gate=gate, w_pre=w_pre, res_scale=-1.5, eps=1e-3)
    _check(H, res, y, w_post, gate, w_pre, -1.5, float(np.float32(1e-3)), r, o, rk, ok)


@pytest.mark.parametrize("H", [64, 1111])
@pytest.mark.parametrize("parts", ["pre", "add", "add_pre", "post", "scale"])
def test_missing_parts(H, parts):
    rng = np.random.default_rng(H)
    y, res = _t(rng.standard_normal((4, H)), "f32"), _t(rng.standard_normal((4, H)), "f32")
    w = _t(rng.standard_normal(H), "f32")
    r, o = torch.empty_like(res), torch.empty_like(res)
    kw = {"pre": dict(w_pre=w), "add": dict(y=y), "add_pre": dict(y=y, w_pre=w), "post": dict(y=y, w_post=w),
          "scale": {}}[parts]
    keep_r, keep_o = parts != "pre", "w_pre" in kw
    block_ops.wd_block_norm(res, r if keep_r else None, o if keep_o else None, res_scale=2.0, **kw)
    _check(H, res, kw.get("y"), kw.get("w_post"), None, kw.get("w_pre"), 2.0, float(np.float32(1e-6)),
           r if keep_r else None, o if keep_o else None, "f32", "f32")


@pytest.mark.parametrize("H,pad", [(128, 8), (128, 1), (2047, 3), (4096, 16)])
def test_strides_and_in_place(H, pad):
    rng = np.random.default_rng(pad)
    T = 6

    def wide(kind, off=0):
        t = torch.full((T, H + pad + off), 9.0, dtype=TYPES[kind], device="cuda")
        t[:, off:off + H] = _t(rng.standard_normal((T, H)), kind)
        return t[:, off:off + H], t
    y, _ = wide("f32", off=1)  # rows off any vector boundary
    res, held = wide("bf16")
    w = _t(rng.standard_normal(H), "f32")
    out, whole = wide("bf16")
    before = res.clone()
    block_ops.wd_block_norm(res, res, out, y=y, w_post=w, w_pre=w)  # res_out is res
    _check(H, before, y, w, None, w, 1.0, float(np.float32(1e-6)), res, out, "bf16", "bf16")
    assert (held[:, H:] == 9).all() and (whole[:, H:] == 9).all()
    over = before.clone()
    block_ops.wd_block_norm(over, None, over, w_pre=w)  # out over res
    _check(H, before, None, None, None, w, 1.0, float(np.float32(1e-6)), None, over, "bf16", "bf16")


def test_zero_rows_infinities_and_large_values():
    H = 256
    res = torch.zeros(4, H, device="cuda")
    w = torch.ones(H, device="cuda")
    res[1] = 1e18  # squares to 1e36: inside FP32
    res[2, 5] = float("inf")
    res[3, 7] = float("nan")
    out = torch.empty_like(res)
    block_ops.wd_block_norm(res, None, out, w_pre=w)
    o = out.cpu().numpy()
    assert (o[0] == 0).all() and np.allclose(o[1], 1.0, rtol=2.0 ** -20)
    assert np.isnan(o[2, 5]) and (np.delete(o[2], 5) == 0).all() and np.isnan(o[3]).all()


def test_another_stream_many_tokens_and_refusals():
    H, T = 64, 70000  # past a 16-bit grid axis
    res = torch.randn(T, H, device="cuda")
    w = torch.rand(H, device="cuda")
    out = torch.empty(T, H, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    block_ops.wd_block_norm(res, None, out, w_pre=w, stream=side)
    side.synchronize()
    pick = torch.tensor([0, 1, 65535, 65536, T - 1], device="cuda")
    _check(H, res[pick], None, None, None, w, 1.0, float(np.float32(1e-6)), None, out[pick], "f32", "f16")
    with pytest.raises(ValueError, match="broadcast"):
        block_ops.wd_block_norm(res, None, out, y=res, gate=w[None, :8], w_pre=w)
    with pytest.raises(TypeError, match="one dtype"):
        block_ops.wd_block_norm(res, None, out, y=res, w_post=w.half(), w_pre=w)
    with pytest.raises(block_ops.WarpDecodeError) as e:
        block_ops.wd_block_norm(res, None, out)
    assert e.value.status == 1
