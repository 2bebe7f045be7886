"""Thin Python binding of the operators around the MoE layer (``include/warp_decode_block.h``).

Every ``wd_*`` function has the name of the C entry point it calls (through
``wd_call``, its arguments as one block), checks
tensor metadata, extracts pointers and raises on a non-OK status, as in
:mod:`ops`. Outputs are the caller's tensors, work is enqueued on ``stream``
(default: the current stream), and nothing synchronises. Tensors may have any
row stride the entry point takes; their last axis is dense.

* ``Fp4Weights``, ``wd_fp4_matvec`` -- projections with MXFP4 weights
* ``Kv4Cache``, ``wd_kv4_append``, ``wd_kv4_gather``, ``wd_kv4_attend`` -- a paged
  KV cache held in MXFP4; ``wd_kv4_attend_chunk`` for several new tokens per sequence
* ``rope_freqs``, ``Rope``, ``wd_rope``, ``wd_kv4_rope_append`` -- rotary positions,
  by themselves and on the way into the cache
* ``wd_block_norm`` -- the norms, gate and residual between two blocks
"""
from __future__ import annotations

import ctypes
import math
from struct import Struct

import torch

from . import ops
from .ops import WarpDecodeError

__all__ = ["Fp4Weights", "Kv4Cache", "kv4_workspace", "wd_fp4_matvec", "wd_kv4_append", "wd_kv4_gather",
           "wd_kv4_attend", "kv4_chunk_workspace", "wd_kv4_attend_chunk", "rope_freqs", "Rope", "wd_rope",
           "wd_kv4_rope_append", "wd_block_norm", "exported_symbols"]

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream() without its Python object


class Fp4Shape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32)]


class Kv4Struct(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class RotationStruct(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("neighbours", ctypes.c_int32), ("magnitude", ctypes.c_double),
                ("turns", ctypes.c_void_p)]


_lib_cache = None  # the entry points read it directly: a call's marshalling is a few us, as long as a small kernel

# wd_call: number and arguments of the entry points of a decode step (q: integers and pointers, d: floats)
_MATVEC, _APPEND, _GATHER, _ATTEND, _NORM = range(5)
_ROPE, _ROPE_APPEND, _CHUNK = 8, 9, 10
_matvec_args = Struct("11q").pack
_token_args = Struct("14q").pack
_attend_args = Struct("9qd8q").pack
_norm_args = Struct("14q2d6q").pack
_rope_args = Struct("11q").pack
_rope_append_args = Struct("20q").pack
_chunk_args = Struct("11qd8q").pack


def lib() -> ctypes.CDLL:
    """The loaded library with these entry points' signatures set."""
    global _lib_cache
    if _lib_cache is None:
        L = ops.lib()
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        fp, kp, rp = ctypes.POINTER(Fp4Shape), ctypes.POINTER(Kv4Struct), ctypes.POINTER(RotationStruct)
        L.wd_fp4_packed_bytes.restype = sz
        L.wd_fp4_packed_bytes.argtypes = [fp, ctypes.c_int]
        L.wd_kv4_cache_bytes.restype = sz
        L.wd_kv4_cache_bytes.argtypes = [kp, ctypes.c_int]
        L.wd_kv4_attend_workspace.restype = sz
        L.wd_kv4_attend_workspace.argtypes = [kp, i32, i32]
        L.wd_kv4_attend_ctas.restype = i32
        L.wd_kv4_attend_ctas.argtypes = [kp, i32, i32, i32, i32]
        L.wd_kv4_attend_chunk_workspace.restype = sz
        L.wd_kv4_attend_chunk_workspace.argtypes = [kp, i32, i32]
        tokens = [kp, vp, vp, i32, i64, i64, i32, vp, i32, vp, vp, i32, vp, vp]
        for name, args in (
                ("wd_fp4_pack_codes", [fp, vp, vp, vp, vp, vp]),
                ("wd_fp4_pack_weights", [fp, vp, i32, i64, vp, vp, vp]),
                ("wd_fp4_matvec", [fp, vp, vp, vp, i32, i64, i32, vp, i32, i64, vp]),
                ("wd_kv4_append", tokens), ("wd_kv4_gather", tokens),
                ("wd_kv4_attend", [kp, vp, i32, i64, i32, i32, vp, i32, vp, f32, i32, vp, i64, vp, vp, sz, vp, vp]),
                ("wd_kv4_attend_chunk", [kp, vp, i32, i64, i32, i32, vp, i32, vp, vp, i32, f32, i32, vp, i64, vp, vp, sz,
                                         vp, vp]),
                ("wd_rope_turns", [i32, vp, vp]),
                ("wd_rope", [rp, vp, i32, i64, i32, i32, i32, vp, vp, i64, vp]),
                ("wd_kv4_rope_append", [kp, rp, vp, i64, i32, vp, i64, *tokens[1:]]),
                ("wd_block_norm", [i32, i32, vp, i32, i64, vp, i32, i64, vp, vp, vp, i32, i64, i32, f32, f32, vp,
                                   i64, vp, i32, i64, vp])):
            fn = getattr(L, name)
            fn.restype = ctypes.c_int
            fn.argtypes = args
        L.wd_call.restype = ctypes.c_int
        L.wd_call.argtypes = [i32, ctypes.c_char_p]
        _lib_cache = L
    return _lib_cache


def exported_symbols() -> list[str]:
    """The entry points include/warp_decode_block.h declares."""
    return ["wd_fp4_packed_bytes", "wd_fp4_pack_codes", "wd_fp4_pack_weights", "wd_fp4_matvec",
            "wd_kv4_cache_bytes", "wd_kv4_append", "wd_kv4_gather", "wd_kv4_attend_workspace",
            "wd_kv4_attend_ctas", "wd_kv4_attend", "wd_kv4_attend_chunk_workspace", "wd_kv4_attend_chunk",
            "wd_rope_turns", "wd_rope", "wd_kv4_rope_append", "wd_block_norm", "wd_call"]


def _check(fn: str, status: int) -> None:
    if status != ops.MOE_OK:
        raise WarpDecodeError(fn, status, lib().moe_last_error().decode())


def _stream(stream, t: torch.Tensor) -> int:
    if stream is None:
        return _raw_stream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _hand_over(stream, *tensors: torch.Tensor) -> None:
    """Let `stream` use tensors of the current stream: it waits for what that one has queued (their memory may still
    be in use there), and their memory is kept until its own work is done."""
    device = tensors[0].device
    if stream is None or device.type != "cuda":
        return
    current = torch.cuda.current_stream(device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return
    stream.wait_stream(current)
    for t in tensors:
        t.record_stream(stream)


def _elsewhere(name: str):
    raise ValueError(f"{name}: not on a GPU")


def _type(t: torch.Tensor, name: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} is not float32, bfloat16 or float16")
    if not t.is_cuda:
        _elsewhere(name)
    return code


def _rows(t: torch.Tensor, shape: tuple, row: int, name: str) -> int:
    """Row stride of a tensor of shape [rows, ...] whose rows are dense, `row` elements each."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return row
    strides = t.stride()
    if len(strides) == 3 and strides[2] == 1 and strides[1] == shape[2]:
        return strides[0]  # (the loop below takes 1 us)
    want = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != want:
            raise ValueError(f"{name}: a row must be dense, got strides {t.stride()}")
        want *= size
    return t.stride(0)


def _ints(t: torch.Tensor, shape: tuple, name: str) -> int:
    if t.dtype is not torch.int32:
        raise TypeError(f"{name}: dtype {t.dtype} is not int32")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        _elsewhere(name)
    return t.data_ptr()


def _flag(t: torch.Tensor) -> int:
    if t.dtype is not torch.int32:
        raise TypeError(f"err_flag: dtype {t.dtype} is not int32")
    if not t.is_cuda or t.numel() == 0:
        raise ValueError("err_flag: expected an element on a GPU")
    return t.data_ptr()


# ---------------------------------------------------------- 4-bit projections --

class Fp4Weights:
    """MXFP4 weights [N, K] on the GPU in the packed layout of warp_decode_block.h.

    `stream` of the two constructors: where they are packed, behind what the current stream has queued (it needs no
    waiting for the inputs, and they may be freed at once). Another stream, the current one too, has to wait for it
    before it uses the weights.
    """

    def __init__(self, N: int, K: int, device="cuda"):
        self.shape = Fp4Shape(N, K)
        self._shape, self._at = ctypes.byref(self.shape), ctypes.addressof(self.shape)
        sizes = [int(lib().wd_fp4_packed_bytes(self._shape, w)) for w in (0, 1)]
        if not all(sizes):
            raise ValueError(f"Fp4Weights: unsupported shape [{N}, {K}] (K % 32 == 0, 32 <= K <= 65536)")
        self.N, self.K = N, K
        self._tensors = tuple(torch.empty(n, dtype=torch.uint8, device=device) for n in sizes)
        self._ptrs = tuple(t.data_ptr() for t in self._tensors)
        self._on_gpu = self._tensors[0].is_cuda

    # read-only: the kernels are given the addresses taken above
    @property
    def codes(self) -> torch.Tensor:
        return self._tensors[0]

    @property
    def scales(self) -> torch.Tensor:
        return self._tensors[1]

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> "Fp4Weights":
        """From an MXFP4 checkpoint: uint8 codes [N, K/2] (even element in the low nibble), scales [N, K/32]."""
        N, K = codes.shape[0], 2 * codes.shape[1]
        for t, shape, name in ((codes, (N, K // 2), "codes"), (scales, (N, K // 32), "scales")):
            if t.dtype != torch.uint8 or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous uint8 {shape}, got {t.dtype} {tuple(t.shape)}")
            if not t.is_cuda:
                _elsewhere(name)
        w = cls(N, K, codes.device)
        _hand_over(stream, codes, scales, *w._tensors)
        _check("wd_fp4_pack_codes", lib().wd_fp4_pack_codes(
            w._shape, codes.data_ptr(), scales.data_ptr(), *w._ptrs, _stream(stream, codes)))
        return w

    @classmethod
    def quantize(cls, w: torch.Tensor, stream=None) -> "Fp4Weights":
        """Quantise w [N, K] (float32, bfloat16 or float16, on the GPU) to MXFP4."""
        if w.dim() != 2:
            raise ValueError(f"w: expected [N, K], got {tuple(w.shape)}")
        kind = _type(w, "w")
        out = cls(w.shape[0], w.shape[1], w.device)
        _hand_over(stream, w, *out._tensors)
        _check("wd_fp4_pack_weights", lib().wd_fp4_pack_weights(
            out._shape, w.data_ptr(), kind, _rows(w, w.shape, w.shape[1], "w"), *out._ptrs, _stream(stream, w)))
        return out

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def wd_fp4_matvec(weights: Fp4Weights, x: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """y[B, N] = x[B, K] W^T; x bfloat16 or float16, y float32, bfloat16 or float16."""
    B, K, N = x.shape[0], weights.K, weights.N
    if not weights._on_gpu:
        _elsewhere("weights")
    codes, scales = weights._ptrs
    status = _lib_cache.wd_call(_MATVEC, _matvec_args(
        weights._at, codes, scales, x.data_ptr(), _type(x, "x"), _rows(x, (B, K), K, "x"), B,
        y.data_ptr(), _type(y, "y"), _rows(y, (B, N), N, "y"), _stream(stream, x)))
    if status:
        _check("wd_fp4_matvec", status)
    return y


# ------------------------------------------------------------- 4-bit KV cache --

class Kv4Cache:
    """One layer's paged KV cache in MXFP4 (four uint8 tensors, layout of warp_decode_block.h)."""

    def __init__(self, pages: int, page_size: int, heads: int, dim: int, device="cuda"):
        self.pages, self.page_size, self.heads, self.dim = pages, page_size, heads, dim
        self.struct = Kv4Struct(pages, page_size, heads, dim)
        self._ref, self._at = ctypes.byref(self.struct), ctypes.addressof(self.struct)
        codes, scales = (int(lib().wd_kv4_cache_bytes(self._ref, w)) for w in (0, 1))
        if not codes:
            raise ValueError(f"Kv4Cache: unsupported sizes: pages {pages}, page_size {page_size} (16 to 256, a power "
                             f"of two), heads {heads}, dim {dim} (64, 128 or 256)")
        self._tensors = tuple(torch.zeros(n, dtype=torch.uint8, device=device) for n in (codes, scales, codes, scales))
        (self.struct.k_codes, self.struct.k_scales, self.struct.v_codes,
         self.struct.v_scales) = (t.data_ptr() for t in self._tensors)
        self._on_gpu = self._tensors[0].is_cuda

    @property
    def tensors(self) -> tuple:
        """K's codes and scales, V's codes and scales. Read-only: the kernels are given their addresses."""
        return self._tensors

    @property
    def nbytes(self) -> int:
        return sum(t.numel() for t in self.tensors)


def _tokens(fn: str, which: int, cache: Kv4Cache, k, v, block_table, seq_lens, cu_new, err_flag, stream) -> None:
    T, S, blocks = k.shape[0], seq_lens.shape[0], block_table.shape[-1]
    if v.dtype != k.dtype:
        raise TypeError(f"v: dtype {v.dtype} differs from k's {k.dtype}")
    if not (cache._on_gpu and v.is_cuda):
        _elsewhere("cache or v")
    row = cache.heads * cache.dim
    shape = (T, cache.heads, cache.dim)
    status = _lib_cache.wd_call(which, _token_args(
        cache._at, k.data_ptr(), v.data_ptr(), _type(k, "k"), _rows(k, shape, row, "k"), _rows(v, shape, row, "v"), T,
        _ints(block_table, (S, blocks), "block_table"), blocks, _ints(seq_lens, (S,), "seq_lens"),
        0 if cu_new is None else _ints(cu_new, (S + 1,), "cu_new"), S,
        0 if err_flag is None else _flag(err_flag), _stream(stream, k)))
    if status:
        _check(fn, status)


def wd_kv4_append(cache: Kv4Cache, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, cu_new: torch.Tensor | None = None,
                  err_flag: torch.Tensor | None = None, stream=None) -> Kv4Cache:
    """Quantise the new tokens k, v [T, heads, dim] into the cache behind seq_lens[s] tokens of each
    sequence; cu_new [S + 1] says which rows are whose (None: one each)."""
    _tokens("wd_kv4_append", _APPEND, cache, k, v, block_table, seq_lens, cu_new, err_flag, stream)
    return cache


def wd_kv4_gather(cache: Kv4Cache, block_table: torch.Tensor, seq_lens: torch.Tensor, k_out: torch.Tensor,
                  v_out: torch.Tensor, cu_new: torch.Tensor | None = None,
                  err_flag: torch.Tensor | None = None, stream=None):
    """The values of the positions that wd_kv4_append with the same arguments writes."""
    _tokens("wd_kv4_gather", _GATHER, cache, k_out, v_out, block_table, seq_lens, cu_new, err_flag, stream)
    return k_out, v_out


def kv4_workspace(cache: Kv4Cache, S: int, q_heads: int) -> torch.Tensor:
    """A workspace for wd_kv4_attend with this cache's sizes: reusable, one per overlapping call."""
    n = int(lib().wd_kv4_attend_workspace(cache._ref, S, q_heads))
    if not n:
        raise ValueError(f"kv4_workspace: S {S} or q_heads {q_heads} (a multiple of {cache.heads}) is unsupported")
    return torch.empty(n, dtype=torch.uint8, device=cache.tensors[0].device)


def wd_kv4_attend(cache: Kv4Cache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  out: torch.Tensor, workspace: torch.Tensor, lse: torch.Tensor | None = None,
                  scale: float | None = None, window: int = 0, err_flag: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """out[S, q_heads, dim]: attention of one query token per sequence over its seq_lens[s] cached keys
    (the last `window` of them, 0 for all); lse [S, q_heads] float32. scale: 1 / sqrt(dim) by default."""
    S, q_heads = q.shape[0], q.shape[1]
    if out.dtype != q.dtype:
        raise TypeError(f"out: dtype {out.dtype} differs from q's {q.dtype}")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (S, q_heads) or not lse.is_contiguous()):
        raise ValueError(f"lse: expected contiguous float32 {(S, q_heads)}, got {lse.dtype} {tuple(lse.shape)}")
    if not (cache._on_gpu and out.is_cuda and workspace.is_cuda and (lse is None or lse.is_cuda)):
        _elsewhere("cache, out, workspace or lse")
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    D, blocks = cache.dim, block_table.shape[-1]
    shape, row = (S, q_heads, D), q_heads * D
    status = _lib_cache.wd_call(_ATTEND, _attend_args(
        cache._at, q.data_ptr(), _type(q, "q"), _rows(q, shape, row, "q"), S, q_heads,
        _ints(block_table, (S, blocks), "block_table"), blocks, _ints(seq_lens, (S,), "seq_lens"),
        D ** -0.5 if scale is None else scale, window, out.data_ptr(), _rows(out, shape, row, "out"),
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        0 if err_flag is None else _flag(err_flag), _stream(stream, q)))
    if status:
        _check("wd_kv4_attend", status)
    return out


def kv4_chunk_workspace(cache: Kv4Cache, T: int, q_heads: int) -> torch.Tensor:
    """A workspace for wd_kv4_attend_chunk with this cache's sizes and up to T tokens: reusable, one per overlapping call."""
    n = int(lib().wd_kv4_attend_chunk_workspace(cache._ref, T, q_heads))
    if not n:
        raise ValueError(f"kv4_chunk_workspace: T {T} or q_heads {q_heads} (a multiple of {cache.heads}) is unsupported")
    return torch.empty(n, dtype=torch.uint8, device=cache.tensors[0].device)


def wd_kv4_attend_chunk(cache: Kv4Cache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                        out: torch.Tensor, workspace: torch.Tensor, cu_new: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, scale: float | None = None, window: int = 0,
                        err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[T, q_heads, dim]: attention of the new tokens q over the cache, which holds them already. block_table, seq_lens
    (without the new tokens) and cu_new are wd_kv4_append's. A token attends to itself and what is before it (to the last
    `window` of these, 0 for all); lse [T, q_heads] float32. scale: 1 / sqrt(dim) by default."""
    T, q_heads, S = q.shape[0], q.shape[1], seq_lens.shape[0]
    if out.dtype != q.dtype:
        raise TypeError(f"out: dtype {out.dtype} differs from q's {q.dtype}")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, q_heads) or not lse.is_contiguous()):
        raise ValueError(f"lse: expected contiguous float32 {(T, q_heads)}, got {lse.dtype} {tuple(lse.shape)}")
    if not (cache._on_gpu and out.is_cuda and workspace.is_cuda and (lse is None or lse.is_cuda)):
        _elsewhere("cache, out, workspace or lse")
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    D, blocks = cache.dim, block_table.shape[-1]
    shape, row = (T, q_heads, D), q_heads * D
    status = _lib_cache.wd_call(_CHUNK, _chunk_args(
        cache._at, q.data_ptr(), _type(q, "q"), _rows(q, shape, row, "q"), T, q_heads,
        _ints(block_table, (S, blocks), "block_table"), blocks, _ints(seq_lens, (S,), "seq_lens"),
        0 if cu_new is None else _ints(cu_new, (S + 1,), "cu_new"), S,
        D ** -0.5 if scale is None else scale, window, out.data_ptr(), _rows(out, shape, row, "out"),
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        0 if err_flag is None else _flag(err_flag), _stream(stream, q)))
    if status:
        _check("wd_kv4_attend_chunk", status)
    return out


# ----------------------------------------------------------- rotary positions --

def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               trained: int | None = None, slow: float = 1.0, fast: float = 32.0) -> torch.Tensor:
    """Radians per position of the rot_dim / 2 pairs: base ** (-2 i / rot_dim), float64 on the CPU. For contexts `factor`
    times as long as those trained on, `scaling` is

    * "linear": every frequency divided by factor (positions interpolated);
    * "base": a larger base, base * factor ** (rot_dim / (rot_dim - 2)): the slowest pair is divided by factor, the fastest stays;
    * "parts": by a pair's turns over the `trained` positions: below `slow` divided by factor, above `fast` left, mixed between.
      Queries and keys are then often multiplied by 0.1 ln(factor) + 1 each (`magnitude` of a Rope).
    """
    if rot_dim < 2 or rot_dim % 2 or not base > 0 or not factor > 0:
        raise ValueError(f"rope_freqs: rot_dim {rot_dim}, base {base} or factor {factor} is unsupported")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim
    if scaling == "base":
        if rot_dim == 2:
            raise ValueError("rope_freqs: a single pair has no other base")
        base *= factor ** (rot_dim / (rot_dim - 2))
    f = base ** -i
    if scaling == "linear":
        return f / factor
    if scaling == "parts":
        if not trained or trained < 1 or not fast > slow:
            raise ValueError("rope_freqs: parts need the trained length, and fast above slow")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        return f * (keep + (1 - keep) / factor)
    if scaling not in (None, "base"):
        raise ValueError(f"rope_freqs: scaling {scaling!r} is not 'linear', 'base' or 'parts'")
    return f


class Rope:
    """A model's rotary positions: pair i of a head's first 2 * len(freqs) elements turns by freqs[i] radians per position
    and is multiplied by magnitude. The pairs are elements i and i + len(freqs), or, `interleaved`, 2 i and 2 i + 1.
    len(freqs) is a multiple of 8, magnitude 0 or from 2^-100 to 65536 in size. Made once: it reads freqs (float32 or float64,
    as rope_freqs makes them) on the host."""

    def __init__(self, freqs: torch.Tensor, interleaved: bool = False, magnitude: float = 1.0, device=None):
        if freqs.dim() != 1 or freqs.dtype not in (torch.float32, torch.float64):
            raise ValueError(f"freqs: expected float32 or float64 [pairs], got {freqs.dtype} {tuple(freqs.shape)}")
        n = freqs.shape[0]
        if n == 0 or n % 8:
            raise ValueError(f"freqs: {n} pairs, not a multiple of 8")
        host = freqs.detach().to(device="cpu", dtype=torch.float64).contiguous()
        turns = torch.empty(n, dtype=torch.int64)
        _check("wd_rope_turns", lib().wd_rope_turns(n, host.data_ptr(), turns.data_ptr()))
        if device is None:
            device = freqs.device if freqs.is_cuda else "cuda"
        self.rot_dim, self.interleaved, self.magnitude = 2 * n, bool(interleaved), float(magnitude)
        self._turns = turns.to(device)
        self.struct = RotationStruct(2 * n, int(self.interleaved), self.magnitude, self._turns.data_ptr())
        self._at = ctypes.addressof(self.struct)
        self._on_gpu = self._turns.is_cuda

    @property
    def turns(self) -> torch.Tensor:
        """The frequencies in turns per position times 2^64, as int64. Read-only: the kernels are given its address."""
        return self._turns


def wd_rope(rope: Rope, x: torch.Tensor, positions: torch.Tensor, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """x [T, heads, dim] (float32, bfloat16 or float16) turned by positions [T] int32 into out (by default x itself).
    Negative positions turn back."""
    out = x if out is None else out
    if out.dtype != x.dtype:
        raise TypeError(f"out: dtype {out.dtype} differs from x's {x.dtype}")
    if not (rope._on_gpu and out.is_cuda):
        _elsewhere("rope or out")
    T, heads, dim = shape = x.shape
    row = heads * dim
    status = _lib_cache.wd_call(_ROPE, _rope_args(
        rope._at, x.data_ptr(), _type(x, "x"), _rows(x, shape, row, "x"), T, heads, dim,
        _ints(positions, (T,), "positions"), out.data_ptr(), _rows(out, shape, row, "out"), _stream(stream, x)))
    if status:
        _check("wd_rope", status)
    return out


def wd_kv4_rope_append(cache: Kv4Cache, rope: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       block_table: torch.Tensor, seq_lens: torch.Tensor, q_out: torch.Tensor | None = None,
                       cu_new: torch.Tensor | None = None, err_flag: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """wd_kv4_append of k turned by its tokens' positions (seq_lens[s] and on) and of v, and q [T, q_heads, dim] turned
    into q_out (by default q itself), which is returned."""
    q_out = q if q_out is None else q_out
    T, S, blocks, q_heads = k.shape[0], seq_lens.shape[0], block_table.shape[-1], q.shape[1]
    if not v.dtype == q.dtype == q_out.dtype == k.dtype:
        raise TypeError(f"q, q_out, k and v must have one dtype, got {q.dtype}, {q_out.dtype}, {k.dtype} and {v.dtype}")
    if not (cache._on_gpu and rope._on_gpu and v.is_cuda and q.is_cuda and q_out.is_cuda):
        _elsewhere("cache, rope, q, q_out or v")
    D = cache.dim
    row, q_row = cache.heads * D, q_heads * D
    shape, q_shape = (T, cache.heads, D), (T, q_heads, D)
    status = _lib_cache.wd_call(_ROPE_APPEND, _rope_append_args(
        cache._at, rope._at, q.data_ptr(), _rows(q, q_shape, q_row, "q"), q_heads, q_out.data_ptr(),
        _rows(q_out, q_shape, q_row, "q_out"), k.data_ptr(), v.data_ptr(), _type(k, "k"), _rows(k, shape, row, "k"),
        _rows(v, shape, row, "v"), T, _ints(block_table, (S, blocks), "block_table"), blocks,
        _ints(seq_lens, (S,), "seq_lens"), 0 if cu_new is None else _ints(cu_new, (S + 1,), "cu_new"), S,
        0 if err_flag is None else _flag(err_flag), _stream(stream, k)))
    if status:
        _check("wd_kv4_rope_append", status)
    return q_out


# ---------------------------------------------------------------- block norms --

def _weight(w: torch.Tensor, H: int, kind: torch.dtype, name: str) -> int:
    if w.dtype is not kind:
        raise TypeError("w_post, w_pre and gate must have one dtype")
    if w.shape != (H,) or not w.is_contiguous():
        raise ValueError(f"{name}: expected contiguous [{H}], got {tuple(w.shape)}")
    if not w.is_cuda:
        _elsewhere(name)
    return w.data_ptr()


def wd_block_norm(res: torch.Tensor, res_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  y: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                  res_scale: float = 1.0, eps: float = 1e-6, stream=None):
    """r' = res_scale * res + gate * norm(y; w_post) into res_out, norm(r'; w_pre) into out: the step
    between two blocks. gate broadcasts from [1 or T, 1 or H]. Returns (res_out, out)."""
    T, H = shape = res.shape
    kind = None
    pp = qp = gp = yp = rp = op = gate_ld = gate_step = yt = yl = rl = ot = ol = 0
    if w_pre is not None:
        kind = w_pre.dtype
        qp = _weight(w_pre, H, kind, "w_pre")
    if w_post is not None:
        kind = kind or w_post.dtype
        pp = _weight(w_post, H, kind, "w_post")
    if gate is not None:
        kind = kind or gate.dtype
        if gate.dtype is not kind:
            raise TypeError("w_post, w_pre and gate must have one dtype")
        rows, cols = gate.shape if gate.dim() == 2 else (0, 0)
        if rows not in (1, T) or cols not in (1, H):
            raise ValueError(f"gate: shape {tuple(gate.shape)} does not broadcast to {(T, H)}")
        if not gate.is_cuda:
            _elsewhere("gate")
        gp = gate.data_ptr()
        gate_ld = gate.stride(0) if rows > 1 else 0
        gate_step = gate.stride(1) if cols > 1 else 0
    if y is not None:
        yp, yt, yl = y.data_ptr(), _type(y, "y"), _rows(y, shape, H, "y")
    if res_out is not None:
        if res_out.dtype != res.dtype:
            raise TypeError(f"res_out: dtype {res_out.dtype} differs from res's {res.dtype}")
        if not res_out.is_cuda:
            _elsewhere("res_out")
        rp, rl = res_out.data_ptr(), _rows(res_out, shape, H, "res_out")
    if out is not None:
        op, ot, ol = out.data_ptr(), _type(out, "out"), _rows(out, shape, H, "out")
    w_type = _TYPES.get(kind, 0)
    if w_type == 0 and kind is not None and kind is not torch.float32:
        raise TypeError(f"w_post, w_pre and gate: dtype {kind} is not float32, bfloat16 or float16")
    status = (_lib_cache or lib()).wd_call(_NORM, _norm_args(
        T, H, res.data_ptr(), _type(res, "res"), H if res.is_contiguous() else _rows(res, shape, H, "res"), yp, yt, yl,
        pp, qp, gp, w_type, gate_ld, gate_step, res_scale, eps, rp, rl, op, ot, ol, _stream(stream, res)))
    if status:
        _check("wd_block_norm", status)
    return res_out, out
