"""The decoder-block operators without a GPU: symbols, sizes and refusals."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from output_centric_expert_gb300 import block_ops, ops

from . import _block_ref as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "warp_decode_block.h")
P = 0x20000  # a fake device address, never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 5


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(wd_[a-z_0-9]+)\s*\(", src)))
    assert declared == sorted(block_ops.exported_symbols())
    for name in declared:
        assert hasattr(block_ops.lib(), name), name


def test_plain_quantiser_rounds_to_nearest_even_and_saturates():
    # one block with scale 1 (largest magnitude in [4, 8)): values and what they become
    v = [7.9, 5, 5.001, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2500001, 0.0, -0.25, -7.0]
    want = [6, 4, 6, 4, 2, 2, 1, 1, 0, 0.5, 0, 0, -6]
    block = np.zeros(32)
    block[:len(v)] = v
    c, s = ref.quantise(block)
    assert s[0] == 127 and np.array_equal(ref.values(c, s)[:len(v)], want)
    assert ref.quantise(np.zeros(32))[1][0] == 0
    block[3] = np.nan
    assert ref.quantise(block)[1][0] == 255 and np.isnan(ref.rounded(block)).all()


def test_packed_sizes():
    L = block_ops.lib()

    def size(N, K, which):
        return L.wd_fp4_packed_bytes(ctypes.byref(block_ops.Fp4Shape(N, K)), which)
    assert size(16, 128, 0) == 1024 and size(16, 128, 1) == 64
    assert size(17, 160, 0) == 4 * 1024 and size(17, 160, 1) == 4 * 64
    assert size(131072, 65536, 0) == 131072 * 65536 // 2  # past 32 bits
    assert size(0, 128, 0) == size(16, 48, 0) == size(16, 0, 0) == size(16, 65568, 0) == size(16, 128, 2) == 0

    def cache(*sizes):
        return [L.wd_kv4_cache_bytes(ctypes.byref(block_ops.Kv4Struct(*sizes)), w) for w in (0, 1)]
    assert cache(3, 16, 2, 128) == [3 * 16 * 2 * 64, 3 * 16 * 2 * 4]
    assert cache(1 << 20, 256, 8, 256)[0] == (1 << 20) * 256 * 8 * 128
    for bad in ((0, 16, 2, 128), (3, 24, 2, 128), (3, 512, 2, 128), (3, 16, 0, 128), (3, 16, 2, 96)):
        assert cache(*bad) == [0, 0]


@pytest.mark.parametrize("change,status", [
    (dict(), 0), (dict(B=0, x=None, y=None), 0),
    (dict(shape=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(B=1, x=None), NULL),
    (dict(B=1, y=None), NULL), (dict(shape=(0, 128)), SHAPE), (dict(shape=(16, 100)), SHAPE),
    (dict(B=-1), SHAPE), (dict(B=1, ldx=120), SHAPE), (dict(B=1, ldy=15), SHAPE),
    (dict(B=1, x_type=0), UNSUPPORTED), (dict(B=1, x_type=7), UNSUPPORTED), (dict(B=1, y_type=3), UNSUPPORTED),
    (dict(codes=P + 16), ALIGN), (dict(B=1, x=P + 8), ALIGN), (dict(B=1, ldx=132), ALIGN),
    (dict(B=1, y=P + 2), ALIGN)])
def test_matvec_refuses_before_launch(change, status):
    a = dict(shape=(16, 128), codes=P, scales=P, x=P, x_type=1, ldx=128, B=0, y=P, y_type=0, ldy=16) | change
    sh = ctypes.byref(block_ops.Fp4Shape(*a["shape"])) if a["shape"] else None
    assert block_ops.lib().wd_fp4_matvec(sh, a["codes"], a["scales"], a["x"], a["x_type"], a["ldx"], a["B"], a["y"],
                                         a["y_type"], a["ldy"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(codes=None), NULL), (dict(w=None), NULL), (dict(ldw=64), SHAPE), (dict(w_type=9), UNSUPPORTED),
    (dict(w=P + 2), ALIGN), (dict(out=P + 4), ALIGN)])
def test_pack_refuses_before_launch(change, status):
    a = dict(codes=P, w=P, w_type=0, ldw=128, out=P) | change
    sh = ctypes.byref(block_ops.Fp4Shape(16, 128))
    out = a["out"] if a["codes"] else None
    assert block_ops.lib().wd_fp4_pack_weights(sh, a["w"], a["w_type"], a["ldw"], out, a["out"], None) == status


@pytest.mark.parametrize("fn", ["wd_kv4_append", "wd_kv4_gather"])
@pytest.mark.parametrize("change,status", [
    (dict(T=0, k=None), 0), (dict(S=0, T=0), 0),
    (dict(k=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(arrays=0), NULL),
    (dict(sizes=(2, 24, 2, 128)), SHAPE), (dict(T=-1), SHAPE), (dict(S=-1), SHAPE), (dict(blocks=0), SHAPE),
    (dict(cu=None), SHAPE), (dict(ldk=248), SHAPE), (dict(type=5), UNSUPPORTED),
    (dict(k=P + 8), ALIGN), (dict(ldv=260), ALIGN), (dict(lens=P + 2), ALIGN), (dict(arrays=P + 8), ALIGN)])
def test_cache_writers_refuse_before_launch(fn, change, status):
    a = dict(sizes=(2, 16, 2, 128), arrays=P, k=P, v=P, type=1, ldk=256, ldv=256, T=3, table=P, blocks=4, lens=P,
             cu=P, S=2) | change
    c = ctypes.byref(block_ops.Kv4Struct(*a["sizes"], *[a["arrays"]] * 4))
    assert getattr(block_ops.lib(), fn)(c, a["k"], a["v"], a["type"], a["ldk"], a["ldv"], a["T"], a["table"],
                                        a["blocks"], a["lens"], a["cu"], a["S"], None, None) == status


def test_append_takes_no_f32():
    c = ctypes.byref(block_ops.Kv4Struct(2, 16, 2, 128, P, P, P, P))
    assert block_ops.lib().wd_kv4_append(c, P, P, 0, 256, 256, 2, P, 4, P, None, 2, None, None) == UNSUPPORTED


@pytest.mark.parametrize("change,status", [
    (dict(S=0, q=None), 0),
    (dict(q=None), NULL), (dict(work=None), NULL), (dict(lens=None), NULL),
    (dict(q_heads=3), SHAPE), (dict(q_heads=0), SHAPE), (dict(window=-1), SHAPE), (dict(ldq=512 - 8), SHAPE),
    (dict(blocks=0), SHAPE), (dict(bytes=64), SHAPE), (dict(type=0), UNSUPPORTED), (dict(q=P + 8), ALIGN),
    (dict(ldo=516), ALIGN), (dict(work=P + 8), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_attend_refuses_before_launch(change, status):
    a = dict(q=P, type=1, ldq=512, S=2, q_heads=4, table=P, blocks=4, lens=P, window=0, out=P, ldo=512, lse=P, work=P,
             bytes=1 << 30) | change
    c = ctypes.byref(block_ops.Kv4Struct(2, 16, 2, 128, P, P, P, P))
    assert block_ops.lib().wd_kv4_attend(c, a["q"], a["type"], a["ldq"], a["S"], a["q_heads"], a["table"], a["blocks"],
                                         a["lens"], 1.0, a["window"], a["out"], a["ldo"], a["lse"], a["work"],
                                         a["bytes"], None, None) == status


def test_call_refuses_what_it_does_not_know():
    L = block_ops.lib()
    assert L.wd_call(5, bytes(8)) == UNSUPPORTED and L.wd_call(-1, bytes(8)) == UNSUPPORTED
    assert L.wd_call(0, None) == NULL


@pytest.mark.parametrize("change,status", [
    ({}, 0), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(res=None), NULL), (dict(ldr=63), SHAPE), (dict(y_type=3), UNSUPPORTED),
    (dict(y=P + 2), ALIGN), (dict(gate=P + 2), ALIGN), (dict(step=2), SHAPE), (dict(ldo=63), SHAPE), (dict(out=None), NULL)])
def test_call_passes_every_argument_on(change, status):
    """The refusals of wd_block_norm, its arguments as a block (T = 0 launches nothing)."""
    a = dict(T=0 if not change else 2, H=64, res=P, ldr=64, y=P, y_type=0, ldy=64, w_post=P, w_pre=P, gate=P, step=1,
             res_out=P, out=P, ldo=64) | change
    args = block_ops._norm_args(a["T"], a["H"], a["res"] or 0, 1, a["ldr"], a["y"], a["y_type"], a["ldy"], a["w_post"],
                                a["w_pre"], a["gate"], 0, 0, a["step"], 1.0, 1e-6, a["res_out"], 64, a["out"] or 0, 1,
                                a["ldo"], 0)
    assert block_ops.lib().wd_call(block_ops._NORM, args) == status


def test_attend_refuses_a_cache_of_too_many_runs():
    c = ctypes.byref(block_ops.Kv4Struct(1 << 27, 256, 2, 128, P, P, P, P))
    assert block_ops.lib().wd_kv4_attend(c, P, 1, 512, 2, 4, P, 4, P, 1.0, 0, P, 512, P, P, 1 << 30, None, None) == SHAPE
    assert b"too many pages" in block_ops.lib().moe_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(T=0, res=None), 0),
    (dict(res=None), NULL), (dict(w_pre=None), NULL), (dict(out=None), NULL), (dict(y=None), NULL),
    (dict(res_out=None, out=None, w_pre=None), NULL),
    (dict(H=0), SHAPE), (dict(H=8193, ldr=9000, ldy=9000, ldo=9000), SHAPE), (dict(T=-1), SHAPE),
    (dict(ldr=63), SHAPE), (dict(ldo=63), SHAPE), (dict(step=2), SHAPE), (dict(y_type=3), UNSUPPORTED),
    (dict(res=P + 1), ALIGN), (dict(y=P + 2), ALIGN), (dict(gate=P + 2), ALIGN)])
def test_norm_refuses_before_launch(change, status):
    a = dict(T=2, H=64, res=P, ldr=64, y=P, y_type=0, ldy=64, w_post=P, w_pre=P, gate=P, step=1, res_out=P, out=P,
             ldo=64) | change
    assert block_ops.lib().wd_block_norm(a["T"], a["H"], a["res"], 1, a["ldr"], a["y"], a["y_type"], a["ldy"],
                                         a["w_post"], a["w_pre"], a["gate"], 0, 0, a["step"], 1.0, 1e-6, a["res_out"],
                                         64, a["out"], 1, a["ldo"], None) == status
    if status:
        assert block_ops.lib().moe_last_error()


def test_binding_checks_tensors():
    with pytest.raises(ValueError, match="row must be dense"):
        block_ops._rows(torch.zeros(4, 6, 2).transpose(1, 2), (4, 2, 6), 12, "x")
    with pytest.raises(ValueError, match="expected shape"):
        block_ops._rows(torch.zeros(4, 6), (4, 5), 5, "x")
    wide = torch.zeros(4, 10, 8)
    assert block_ops._rows(wide[:, 2:5], (4, 3, 8), 24, "x") == 80
    assert block_ops._rows(wide[:1, 2:5], (1, 3, 8), 24, "x") >= 24  # one row: its stride is not used
    with pytest.raises(TypeError, match="int32"):
        block_ops._ints(torch.zeros(3, dtype=torch.int64), (3,), "seq_lens")
    with pytest.raises(TypeError, match="dtype"):
        block_ops._type(torch.zeros(3, dtype=torch.float64), "x")
    assert ops.status_string(SHAPE) == "unsupported shape"
