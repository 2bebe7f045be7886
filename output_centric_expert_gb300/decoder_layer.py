"""A decoder layer around the MoE layer, on caller-held state: decode steps, and chunks of new tokens.

The whole layer for the B sequences of a batch, one new token each (`step`):

    a = norm(res; attn_pre)                       wd_block_norm
    q, k, v = a W_qkv^T                           wd_fp4_matvec (MXFP4 weights)
    q, k rotated by their positions               torch
    k, v into the paged MXFP4 cache               wd_kv4_append
    s = attention of q over the cache             wd_kv4_attend
    o = s W_o^T                                   wd_fp4_matvec
    res' = res + norm(o; attn_post), m = norm(res'; moe_pre)      wd_block_norm
    y = MoE(m), routed from m W_router^T          ops.moe_layer_routed (MXFP8 weights)
    res'' = res' + gate * norm(y; moe_post)       wd_block_norm

With a `Rope` the rotation is part of the append (wd_kv4_rope_append), and `extend` takes several
new tokens of each sequence through the layer: a prompt, a chunk of one or a draft, attended to by
wd_kv4_attend_chunk.

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
    sequence's length before the step, below `max_positions`, for which the rotations are tabled. With `rope` the
    positions have no such bound and no tables (`max_positions` may be None, `rope_base` is not used), and `extend`
    takes up to `max_batch` tokens."""

    def __init__(self, weights: LayerWeights, cache: block_ops.Kv4Cache, q_heads: int, max_batch: int,
                 max_positions: int | None, rope_base: float = 10000.0, eps: float = 1e-6,
                 rope: block_ops.Rope | None = None):
        shape, dim, kv = weights.moe.shape, cache.dim, cache.heads
        H = shape.H
        if weights.qkv.N != (q_heads + 2 * kv) * dim or weights.qkv.K != H:
            raise ValueError(f"qkv: expected [{(q_heads + 2 * kv) * dim}, {H}], got [{weights.qkv.N}, {weights.qkv.K}]")
        if weights.o.N != H or weights.o.K != q_heads * dim:
            raise ValueError(f"o: expected [{H}, {q_heads * dim}], got [{weights.o.N}, {weights.o.K}]")
        if rope is None and max_positions is None:
            raise ValueError("max_positions: expected the tables' length, or a rope")
        if rope is not None and rope.rot_dim > dim:
            raise ValueError(f"rope: turns {rope.rot_dim} elements of heads of {dim}")
        self.w, self.cache, self.q_heads, self.eps, self.rope = weights, cache, q_heads, eps, rope
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
        if rope is not None:
            self.chunk_workspace = block_ops.kv4_chunk_workspace(cache, max_batch, q_heads)
            return
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
        cache or no rotation sets bit 0 of err_flag, and its output does not count. Without rows nothing is done."""
        B = res.shape[0]
        if B == 0:
            return res
        q, k, v, turned = self._project(res)
        if self.rope is None:
            self._rotate(turned, self._positions(seq_lens, err_flag))
            block_ops.wd_kv4_append(self.cache, k, v, block_table, seq_lens, err_flag=err_flag)
        else:
            block_ops.wd_kv4_rope_append(self.cache, self.rope, q, k, v, block_table, seq_lens, err_flag=err_flag)
        lens = torch.add(seq_lens, 1, out=self.lens[:B])
        block_ops.wd_kv4_attend(self.cache, q, block_table, lens, self.attn[:B], self.workspace, err_flag=err_flag)
        return self._behind_attention(res, err_flag)

    def extend(self, res: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, cu_new: torch.Tensor,
               err_flag: torch.Tensor | None = None) -> torch.Tensor:
        """Several new tokens of each sequence through the layer: res [T, H] (bfloat16 or float32), rows cu_new[s] to
        cu_new[s + 1] - 1 of sequence s, is updated in place and returned. seq_lens [S]: tokens that the cache holds
        before the call. Rows behind cu_new[S] (padding; finite) come out undefined, but finite, and touch nothing else. The layer needs a
        rope. err_flag as for a step. Without rows nothing is done."""
        if self.rope is None:
            raise ValueError("extend: the layer has no rope")
        T = res.shape[0]
        if T > self.a.shape[0]:
            raise ValueError(f"extend: {T} tokens, the layer's buffers hold {self.a.shape[0]}")
        if T == 0:
            return res
        q, k, v, _ = self._project(res)
        block_ops.wd_kv4_rope_append(self.cache, self.rope, q, k, v, block_table, seq_lens, cu_new=cu_new, err_flag=err_flag)
        attn = self.attn[:T].zero_()  # padding rows are not written: what an earlier call left there could be NaN
        block_ops.wd_kv4_attend_chunk(self.cache, q, block_table, seq_lens, attn, self.chunk_workspace, cu_new,
                                      err_flag=err_flag)
        return self._behind_attention(res, err_flag)

    def _project(self, res: torch.Tensor):
        """q, k, v and q and k together, views of the layer's buffer."""
        w, B, n = self.w, res.shape[0], self.q_heads
        a = self.a[:B]
        block_ops.wd_block_norm(res, None, a, w_pre=w.attn_pre, eps=self.eps)
        heads = block_ops.wd_fp4_matvec(w.qkv, a, self.qkv[:B]).view(B, -1, self.cache.dim)
        both = heads[:, :n + self.cache.heads]
        return heads[:, :n], heads[:, n:n + self.cache.heads], heads[:, n + self.cache.heads:], both

    def _behind_attention(self, res: torch.Tensor, err_flag: torch.Tensor | None) -> torch.Tensor:
        w, B = self.w, res.shape[0]
        m, o, y = self.m[:B], self.o[:B], self.y[:B]
        block_ops.wd_fp4_matvec(w.o, self.attn[:B].view(B, -1), o)
        block_ops.wd_block_norm(res, res, m, y=o, w_post=w.attn_post, w_pre=w.moe_pre, eps=self.eps)
        logits = torch.mm(m.float(), w.router.T)
        ops.moe_layer_routed(w.moe, m, logits, self.h[:B], y, self.ids[:B], self.wts[:B], err_flag)
        block_ops.wd_block_norm(res, res, y=y, w_post=w.moe_post, gate=w.moe_gate, eps=self.eps)
        return res
