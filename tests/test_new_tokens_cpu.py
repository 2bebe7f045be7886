"""Rotary positions, the append with rotation and the attention of chunks without a GPU: frequencies and refusals."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops

from .test_block_devices_cpu import _gpu, _refuses

P = 0x20000  # a fake device address, never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 5
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)


def _turns(freqs):
    f, out = np.array(freqs, np.float64), np.zeros(len(freqs), np.uint64)
    status = block_ops.lib().wd_rope_turns(len(f), f.ctypes.data, out.ctypes.data)
    return status, out


def test_turns_are_exact_to_two_units():
    freqs = list(block_ops.rope_freqs(128).numpy()) + list(block_ops.rope_freqs(64, base=5e6).numpy()) + \
        [0.0, 1e-300, 2 * math.pi, math.pi, 1.0, -1.0, -0.3, 6.5, 1000.0, -65536.0, 65535.9, 5e-11]
    status, got = _turns(freqs)
    assert status == 0
    for f, t in zip(freqs, got):
        want = round(Fraction(float(f)) / (2 * PI) * 2 ** 64) % 2 ** 64
        off = (int(t) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2, f


@pytest.mark.parametrize("freqs,status", [([float("nan")], UNSUPPORTED), ([float("inf")], UNSUPPORTED), ([1.0, 65537.0], UNSUPPORTED), ([], 0)])
def test_turns_refuse(freqs, status):
    assert _turns(freqs)[0] == status
    assert block_ops.lib().wd_rope_turns(-1, P, P) == SHAPE and block_ops.lib().wd_rope_turns(1, None, P) == NULL


def test_frequencies():
    f = block_ops.rope_freqs(64)
    assert f.dtype == torch.float64 and torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-15)
    assert torch.allclose(block_ops.rope_freqs(64, scaling="linear", factor=4.0), f / 4, rtol=1e-15)
    g = block_ops.rope_freqs(64, scaling="base", factor=4.0)
    assert g[0] == 1 and abs(g[-1] / f[-1] * 4 - 1) < 1e-13
    h = block_ops.rope_freqs(64, scaling="parts", factor=8.0, trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(h[turns >= 32], f[turns >= 32]) and torch.allclose(h[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (h[between] < f[between]).all() and (h[between] > f[between] / 8).all()
    for bad in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=64, base=0.0), dict(rot_dim=64, factor=0.0), dict(rot_dim=64, scaling="parts"),
                dict(rot_dim=64, scaling="other"), dict(rot_dim=2, scaling="base"), dict(rot_dim=64, scaling="parts", trained=10, fast=1.0)):
        with pytest.raises(ValueError):
            block_ops.rope_freqs(**bad)


def test_rope_objects():
    r = block_ops.Rope(block_ops.rope_freqs(32), interleaved=True, magnitude=1.5, device="cpu")
    assert (r.rot_dim, r.struct.rot_dim, r.struct.neighbours, r.struct.magnitude) == (32, 32, 1, 1.5)
    assert r.struct.turns == r.turns.data_ptr() and np.array_equal(r.turns.numpy().view(np.uint64), _turns(block_ops.rope_freqs(32).numpy())[1])
    with pytest.raises(AttributeError):
        r.turns = r.turns.clone()
    for bad in (block_ops.rope_freqs(18), torch.zeros(0), torch.zeros(2, 8), torch.zeros(8, dtype=torch.int64)):
        with pytest.raises(ValueError, match="freqs"):
            block_ops.Rope(bad, device="cpu")
    with pytest.raises(block_ops.WarpDecodeError):
        block_ops.Rope(torch.full((8,), float("nan")), device="cpu")


def _rotation(rot=64, magnitude=1.0, turns=P):
    return ctypes.byref(block_ops.RotationStruct(rot, 0, magnitude, turns))


@pytest.mark.parametrize("change,status", [
    (dict(T=0, x=None), 0), (dict(heads=0, x=None, out=None), 0),
    (dict(r=None), NULL), (dict(x=None), NULL), (dict(out=None), NULL), (dict(pos=None), NULL), (dict(r=_rotation(turns=None)), NULL),
    (dict(T=-1), SHAPE), (dict(heads=-1), SHAPE), (dict(dim=60), SHAPE), (dict(dim=8), SHAPE), (dict(dim=1032, ldx=4128, ldo=4128), SHAPE),
    (dict(r=_rotation(8)), SHAPE), (dict(r=_rotation(24)), SHAPE), (dict(r=_rotation(80)), SHAPE), (dict(ldx=248), SHAPE), (dict(ldo=248), SHAPE),
    (dict(heads=20000, ldx=1 << 30, ldo=1 << 30), SHAPE), (dict(out=P, ldo=264), SHAPE),
    (dict(type=3), UNSUPPORTED), (dict(r=_rotation(magnitude=float("inf"))), UNSUPPORTED), (dict(r=_rotation(magnitude=float("nan"))), UNSUPPORTED),
    (dict(x=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(ldx=260), ALIGN), (dict(pos=P + 2), ALIGN), (dict(r=_rotation(turns=P + 4)), ALIGN)])
def test_rope_refuses_before_launch(change, status):
    a = dict(r=_rotation(), x=P, type=1, ldx=256, T=2, heads=4, dim=64, pos=P, out=P + 4096, ldo=256) | change
    assert block_ops.lib().wd_rope(*a.values(), None) == status


APPEND = dict(sizes=(2, 16, 2, 128), arrays=P, r=_rotation(), q=P, ldq=1024, q_heads=8, q_out=P + 65536, ldqo=1024, k=P, v=P, type=1,
              ldk=256, ldv=256, T=3, table=P, blocks=4, lens=P, cu=P, S=2, err=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=0, k=None, q=None), 0), (dict(S=0, T=0), 0),
    (dict(k=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL), (dict(r=None), NULL), (dict(table=None), NULL), (dict(arrays=0), NULL),
    (dict(sizes=(2, 24, 2, 128)), SHAPE), (dict(T=-1), SHAPE), (dict(cu=None), SHAPE), (dict(ldk=248), SHAPE), (dict(ldq=1016), SHAPE),
    (dict(ldqo=1016), SHAPE), (dict(q_heads=-1), SHAPE), (dict(q_heads=8193, ldq=1 << 30, ldqo=1 << 30), SHAPE), (dict(q_out=P, ldqo=1032), SHAPE),
    (dict(r=_rotation(144)), SHAPE), (dict(type=0), UNSUPPORTED), (dict(q=P + 8), ALIGN), (dict(ldq=1028), ALIGN), (dict(q_out=P + 8), ALIGN),
    (dict(v=P + 8), ALIGN), (dict(lens=P + 2), ALIGN), (dict(err=P + 1), ALIGN)])
def test_rope_append_refuses_before_launch(change, status):
    a = dict(APPEND) | change
    c = ctypes.byref(block_ops.Kv4Struct(*a.pop("sizes"), *[a.pop("arrays")] * 4))
    assert block_ops.lib().wd_kv4_rope_append(c, *a.values(), None) == status


CHUNK = dict(q=P, type=1, ldq=512, T=3, q_heads=4, table=P, blocks=4, lens=P, cu=P, S=2, scale=1.0, window=0, out=P, ldo=512, lse=P, work=P,
             bytes=1 << 40, err=None)


@pytest.mark.parametrize("change,status", [
    (dict(T=0, q=None), 0), (dict(S=0, T=0, q=None), 0), (dict(S=0), 0),
    (dict(q=None), NULL), (dict(work=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(out=None), NULL),
    (dict(q_heads=3), SHAPE), (dict(q_heads=0), SHAPE), (dict(window=-1), SHAPE), (dict(ldq=504), SHAPE), (dict(ldo=504), SHAPE),
    (dict(blocks=0), SHAPE), (dict(bytes=0), SHAPE), (dict(cu=None), SHAPE), (dict(T=-1), SHAPE), (dict(S=-1), SHAPE),
    (dict(blocks=1 << 27), SHAPE), (dict(T=1 << 29), SHAPE),
    (dict(type=0), UNSUPPORTED), (dict(q=P + 8), ALIGN), (dict(ldo=516), ALIGN), (dict(work=P + 8), ALIGN), (dict(lse=P + 2), ALIGN),
    (dict(cu=P + 1), ALIGN)])
def test_chunk_refuses_before_launch(change, status):
    a = dict(CHUNK) | change
    c = ctypes.byref(block_ops.Kv4Struct(2, 16, 2, 128, P, P, P, P))
    assert block_ops.lib().wd_kv4_attend_chunk(c, *a.values(), None) == status


def test_chunk_workspace():
    def size(T, heads, *sizes):
        return block_ops.lib().wd_kv4_attend_chunk_workspace(ctypes.byref(block_ops.Kv4Struct(*sizes)), T, heads)
    assert 0 < size(1, 4, 2, 16, 2, 128) <= size(1 << 20, 4, 2, 16, 2, 128) < 1 << 30
    assert size(1, 3, 2, 16, 2, 128) == size(-1, 4, 2, 16, 2, 128) == size(1, 4, 2, 16, 2, 96) == size(1, 0, 2, 16, 2, 128) == 0


SHAPE128 = block_ops.Kv4Struct(2, 16, 2, 128, P, P, P, P)
ROTATION = block_ops.RotationStruct(64, 0, 1.0, P)
CALLS = {  # arguments that launch nothing, and which of them have 32 bits
    "rope": (block_ops._ROPE, block_ops._rope_args, [ctypes.addressof(ROTATION), P, 1, 256, 0, 4, 64, P, P, 256, 0], [2, 4, 5, 6]),
    "append": (block_ops._ROPE_APPEND, block_ops._rope_append_args,
               [ctypes.addressof(SHAPE128), ctypes.addressof(ROTATION), P, 1024, 8, P, 1024, P, P, 1, 256, 256, 0, P, 4, P, P, 0, 0, 0], [4, 9, 12, 14, 17]),
    "chunk": (block_ops._CHUNK, block_ops._chunk_args,
              [ctypes.addressof(SHAPE128), P, 1, 512, 0, 4, P, 4, P, P, 0, 1.0, 7, P, 512, P, P, 1 << 40, 0, 0], [2, 4, 5, 7, 10, 12])}


@pytest.mark.parametrize("name,at", [(n, None) for n in CALLS] + [(n, at) for n, c in CALLS.items() for at in c[3]])
def test_arguments_as_a_block(name, at):
    which, pack, args, _ = CALLS[name]
    if at is None:
        assert block_ops.lib().wd_call(which, pack(*args)) == 0
        return
    for past in (1 << 32, -(1 << 32), 1 << 62):
        wide = list(args)
        wide[at] += past
        assert block_ops.lib().wd_call(which, pack(*wide)) == SHAPE
        assert b"32 bits" in block_ops.lib().moe_last_error()


BF16, INT = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)


@pytest.mark.parametrize("spoiled", ["rope", "x", "positions", "out"])
def test_rope_tensors_elsewhere(spoiled):
    r = block_ops.Rope(block_ops.rope_freqs(16), device="cpu")
    r._on_gpu = spoiled != "rope"
    _refuses(block_ops.wd_rope, dict(rope=r, x=torch.zeros(2, 1, 16, **BF16), positions=torch.zeros(2, **INT), out=torch.zeros(2, 1, 16, **BF16)), [spoiled])


@pytest.mark.parametrize("spoiled", ["cache", "rope", "q", "q_out", "k", "v", "block_table", "seq_lens", "cu_new", "err_flag"])
def test_rope_append_tensors_elsewhere(spoiled):
    r = block_ops.Rope(block_ops.rope_freqs(64), device="cpu")
    c = block_ops.Kv4Cache(2, 16, 1, 64, device="cpu")
    c._on_gpu, r._on_gpu = spoiled != "cache", spoiled != "rope"
    x = [torch.zeros(2, 1, 64, **BF16) for _ in range(4)]
    _refuses(block_ops.wd_kv4_rope_append, dict(cache=c, rope=r, q=x[0], k=x[1], v=x[2], block_table=torch.zeros(1, 2, **INT), seq_lens=torch.zeros(1, **INT),
                                                q_out=x[3], cu_new=torch.zeros(2, **INT), err_flag=torch.zeros(1, **INT)), [spoiled])


@pytest.mark.parametrize("spoiled", ["cache", "q", "block_table", "seq_lens", "out", "workspace", "cu_new", "lse", "err_flag"])
def test_chunk_tensors_elsewhere(spoiled):
    c = block_ops.Kv4Cache(2, 16, 1, 64, device="cpu")
    c._on_gpu = spoiled != "cache"
    _refuses(block_ops.wd_kv4_attend_chunk,
             dict(cache=c, q=torch.zeros(2, 2, 64, **BF16), block_table=torch.zeros(1, 2, **INT), seq_lens=torch.zeros(1, **INT), out=torch.zeros(2, 2, 64, **BF16),
                  workspace=torch.zeros(1 << 20, dtype=torch.uint8), cu_new=torch.zeros(2, **INT), lse=torch.zeros(2, 2), err_flag=torch.zeros(1, **INT)), [spoiled])


def test_gpu_stand_in():
    assert _gpu(torch.zeros(1)).is_cuda
