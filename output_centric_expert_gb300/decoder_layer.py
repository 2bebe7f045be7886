"""One decode step of a decoder layer around the MoE layer, on caller-held state.

The whole layer for the B sequences of a batch, one new token each:

    a = norm(res; attn_pre)                       wd_block_norm
    q, k, v = a W_qkv^T                           wd_fp4_matvec (MXFP4 weights)
    q, k rotated by their positions               torch
    k, v into the paged MXFP4 cache               wd_kv4_append
    s = attention of q over the cache             wd_kv4_attend
    o = s W_o^T                                   wd_fp4_matvec
    res' = res + norm(o; attn_post), m = norm(res'; moe_pre)      wd_block_norm
    y = MoE(m), routed from m W_router^T          ops.moe_layer_routed (MXFP8 weights)
    res'' = res' + gate * norm(y; moe_post)       wd_block_norm

Every buffer is allocated once for the largest batch and every call goes to the
current stream, so a step neither allocates device memory (but for torch's rotation
and router product) nor synchronises.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import block_ops, ops


@dataclass
class LayerWeights:
    """Weights of one layer. The norms are [H]; post norms and the gate may be None."""

    qkv: block_ops.Fp4Weights  # [(q_heads + 2 kv_heads) * dim, H]
    o: block_ops.Fp4Weights    # [H, q_heads * dim]
    router: torch.Tensor       # [E, H] float32
    moe: ops.DeviceWeights
    attn_pre: torch.Tensor
    moe_pre: torch.Tensor
    attn_post: torch.Tensor | None = None
    moe_post: torch.Tensor | None = None
    moe_gate: torch.Tensor | None = None  # [1, H] or [B, 1]


class DecoderLayer:
    """A layer with its step's buffers. `cache` is the layer's own KV cache. A token's position is its
    sequence's length before the step, below `max_positions`, for which the rotations are tabled."""

    def __init__(self, weights: LayerWeights, cache: block_ops.Kv4Cache, q_heads: int, max_batch: int,
                 max_positions: int, rope_base: float = 10000.0, eps: float = 1e-6):
        shape, dim, kv = weights.moe.shape, cache.dim, cache.heads
        H = shape.H
        if weights.qkv.N != (q_heads + 2 * kv) * dim or weights.qkv.K != H:
            raise ValueError(f"qkv: expected [{(q_heads + 2 * kv) * dim}, {H}], got [{weights.qkv.N}, {weights.qkv.K}]")
        if weights.o.N != H or weights.o.K != q_heads * dim:
            raise ValueError(f"o: expected [{H}, {q_heads * dim}], got [{weights.o.N}, {weights.o.K}]")
        self.w, self.cache, self.q_heads, self.eps = weights, cache, q_heads, eps
        device = weights.router.device

        def buf(*size, dtype=torch.bfloat16):
            return torch.empty(max_batch, *size, dtype=dtype, device=device)
        self.a, self.m = buf(H), buf(H)
        self.qkv = buf(weights.qkv.N)
        self.attn, self.o = buf(q_heads, dim), buf(H, dtype=torch.float32)
        self.h = buf(shape.top_k, shape.I)
        self.y = buf(H, dtype=torch.float32)
        self.ids, self.wts = buf(shape.top_k, dtype=torch.int32), buf(shape.top_k, dtype=torch.float32)
        self.lens = torch.empty(max_batch, dtype=torch.int32, device=device)
        self.workspace = block_ops.kv4_workspace(cache, max_batch, q_heads)
        freq = rope_base ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float32) / dim)
        angle = torch.arange(max_positions, device=device, dtype=torch.float32)[:, None] * freq
        self.cos, self.sin = angle.cos(), angle.sin()

    def _positions(self, seq_lens: torch.Tensor, err_flag: torch.Tensor | None) -> torch.Tensor:
        """The tokens' rows in the rotations' tables. A length outside them takes the nearest and sets bit 0 of
        err_flag, as the operators do with one outside the cache: nothing indexes a table with it."""
        pos = seq_lens.clamp(0, self.cos.shape[0] - 1)
        if err_flag is not None:
            err_flag.bitwise_or_((pos != seq_lens).any())
        return pos

    def _rotate(self, x: torch.Tensor, pos: torch.Tensor) -> None:
        """Rotate the halves of x [B, heads, dim] by its tokens' positions, in place."""
        cos, sin = self.cos[pos][:, None], self.sin[pos][:, None]
        lo, hi = x.float().chunk(2, -1)
        x.copy_(torch.cat((lo * cos - hi * sin, hi * cos + lo * sin), -1))

    def step(self, res: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
             err_flag: torch.Tensor | None = None) -> torch.Tensor:
        """One token of each sequence through the layer: res [B, H] (bfloat16 or float32) is updated in
        place and returned. seq_lens [B]: tokens that the cache holds before the step. What has no place in the
        cache or no rotation sets bit 0 of err_flag, and its output does not count."""
        w, B, D, n = self.w, res.shape[0], self.cache.dim, self.q_heads
        a, m, o, y = self.a[:B], self.m[:B], self.o[:B], self.y[:B]
        block_ops.wd_block_norm(res, None, a, w_pre=w.attn_pre, eps=self.eps)
        heads = block_ops.wd_fp4_matvec(w.qkv, a, self.qkv[:B]).view(B, -1, D)
        q, k, v = heads[:, :n], heads[:, n:n + self.cache.heads], heads[:, n + self.cache.heads:]
        self._rotate(heads[:, :n + self.cache.heads], self._positions(seq_lens, err_flag))
        block_ops.wd_kv4_append(self.cache, k, v, block_table, seq_lens, err_flag=err_flag)
        lens = torch.add(seq_lens, 1, out=self.lens[:B])
        block_ops.wd_kv4_attend(self.cache, q, block_table, lens, self.attn[:B], self.workspace, err_flag=err_flag)
        block_ops.wd_fp4_matvec(w.o, self.attn[:B].view(B, n * D), o)
        block_ops.wd_block_norm(res, res, m, y=o, w_post=w.attn_post, w_pre=w.moe_pre, eps=self.eps)
        logits = torch.mm(m.float(), w.router.T)
        ops.moe_layer_routed(w.moe, m, logits, self.h[:B], y, self.ids[:B], self.wts[:B], err_flag)
        block_ops.wd_block_norm(res, res, y=y, w_post=w.moe_post, gate=w.moe_gate, eps=self.eps)
        return res
