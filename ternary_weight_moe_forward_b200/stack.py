"""A stack of decoder layers: attention sublayer, then the ternary MoE layer.

The model's layers are windowed (512 tokens) and global in a 3:1 ratio
("linlog.top/article/1232", section 架构设计, model table); each is

    resid += out(attention(rope(norm(qkv(RMSNorm(resid))))))
    resid += MoE(RMSNorm(resid))

with the residual stream fp32 [T][d_model], int8 projections, bf16 heads and
keys and values cached in 4 bits.  The MoE half is maple_moe_stack_forward.
Everything runs on the current stream without synchronising, and a decode step
may be captured into a CUDA graph.  A stack is used from one stream at a time
(its MoE handles are).

Projections, head counts, norms of the heads and the cache's format are this
library's own choices: the pages do not give them.
"""
from __future__ import annotations

import torch

from . import maple_moe_stack_forward
from .attention import cached_attention, int8_linear, kv_pages, kv_read, prompt_attention, qk_norm_rope

__all__ = ["AttentionLayer", "DecoderStack"]


class AttentionLayer:
    """The attention sublayer with its own cache.

    weights: qkv int8 [(heads + 2 kv_heads) head_dim][d_model], alpha_qkv fp32 (one scale per output channel), out int8
    [d_model][heads head_dim], alpha_out fp32, and optionally q_norm, k_norm fp32 [head_dim] (numpy or torch).  window:
    positions that a query sees (0: all before it).  num_pages x page_size tokens fit its cache.
    """

    def __init__(self, d_model: int, heads: int, kv_heads: int, head_dim: int, weights: dict, num_pages: int, window: int = 0,
                 page_size: int = 64, rotary_dim: int | None = None, theta: float = 10000.0, device="cuda"):
        def dev(name, dtype, shape):
            if weights.get(name) is None:
                if name in ("q_norm", "k_norm"):
                    return None
                raise ValueError(f"{name} is missing")
            t = torch.as_tensor(weights[name]).detach().to(device=device, dtype=dtype).contiguous()
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
            return t

        n = (heads + 2 * kv_heads) * head_dim
        self.d_model, self.heads, self.kv_heads, self.head_dim, self.window = d_model, heads, kv_heads, head_dim, window
        self.qkv, self.alpha_qkv = dev("qkv", torch.int8, (n, d_model)), dev("alpha_qkv", torch.float32, (n,))
        self.out, self.alpha_out = dev("out", torch.int8, (d_model, heads * head_dim)), dev("alpha_out", torch.float32, (d_model,))
        self.q_norm, self.k_norm = dev("q_norm", torch.float32, (head_dim,)), dev("k_norm", torch.float32, (head_dim,))
        rot = head_dim if rotary_dim is None else rotary_dim
        self.inv_freq = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))
        self.pages = kv_pages(num_pages, kv_heads, head_dim, page_size, device)
        self.page_size = page_size
        self.flags = torch.zeros(1, dtype=torch.int32, device=device)

    def _heads(self, resid: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor):
        """Projected, normed and rotated heads; the new keys and values are in the cache afterwards."""
        H, Hkv, d = self.heads, self.kv_heads, self.head_dim
        qkv = int8_linear(resid, self.qkv, self.alpha_qkv, normalise=True, out_dtype=torch.bfloat16, flags=self.flags)
        q, k, v = qkv.view(-1, H + 2 * Hkv, d).split((H, Hkv, Hkv), 1)
        q, k = qk_norm_rope(q, k, positions, self.inv_freq, self.q_norm, self.k_norm, v=v, pages=self.pages, slots=slots,
                            flags=self.flags, page_size=self.page_size)
        return q, k, v

    def _project(self, heads: torch.Tensor, resid: torch.Tensor) -> None:
        int8_linear(heads.flatten(1), self.out, self.alpha_out, resid=resid, out=resid, flags=self.flags)

    def prompt(self, resid: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor, cu: torch.Tensor, max_len: int,
               context: tuple | None = None) -> torch.Tensor:
        """Packed prompts (cu int32 [B+1]); resid [T][d_model] is updated in place.

        context = (slots int64 [Tk], cu_k int32 [B+1]) continues sequences whose beginning is cached already: the slots
        of all of their tokens in order, the new ones last; keys and values are then read from the cache.
        """
        q, k, v = self._heads(resid, positions, slots)
        cu_k = cu
        if context is not None:
            k, v = kv_read(self.pages, context[0], self.head_dim, dtype=q.dtype, flags=self.flags, page_size=self.page_size)
            cu_k = context[1]
        self._project(prompt_attention(q, k, v, cu, cu_k, max_len, window=self.window, flags=self.flags,
                                       out=torch.zeros_like(q)), resid)
        return resid

    def decode(self, resid: torch.Tensor, positions: torch.Tensor, slots: torch.Tensor, block_table: torch.Tensor,
               lens: torch.Tensor) -> torch.Tensor:
        """One new token per sequence (lens counts it); resid [B][d_model] is updated in place."""
        q, _, _ = self._heads(resid, positions, slots)
        self._project(cached_attention(q, self.pages, block_table, lens, window=self.window, flags=self.flags,
                                       page_size=self.page_size), resid)
        return resid


class DecoderStack:
    """Layers as (AttentionLayer, Layer) pairs of one d_model, run one after the other on a residual stream."""

    def __init__(self, layers):
        self.layers = list(layers)
        for attn, moe in self.layers:
            if attn.d_model != moe.shape.d_model:
                raise ValueError("the halves of a layer differ in d_model")

    def _run(self, resid: torch.Tensor, step) -> torch.Tensor:
        if resid.dtype is not torch.float32 or resid.dim() != 2 or not resid.is_contiguous():
            raise ValueError("resid must be contiguous fp32 [T][d_model]")
        # (before anything is changed: a layer that refuses a call has a residual and a cache from the layers before it)
        most = min((moe.max_tokens for _, moe in self.layers), default=resid.shape[0])
        if resid.shape[0] > most:
            raise ValueError(f"{resid.shape[0]} tokens, but a layer takes at most {most}")
        stream = torch.cuda.current_stream(resid.device).cuda_stream
        with torch.cuda.device(resid.device):
            for attn, moe in self.layers:
                step(attn)
                maple_moe_stack_forward([moe.handle], resid, resid.shape[0], stream)
        return resid

    def prompt(self, resid, positions, slots, cu, max_len, context=None) -> torch.Tensor:
        """All layers over packed prompts (arguments of AttentionLayer.prompt); resid is updated in place."""
        return self._run(resid, lambda attn: attn.prompt(resid, positions, slots, cu, max_len, context))

    def decode(self, resid, positions, slots, block_table, lens) -> torch.Tensor:
        """All layers over one new token per sequence (arguments of AttentionLayer.decode); resid is updated in place."""
        return self._run(resid, lambda attn: attn.decode(resid, positions, slots, block_table, lens))

    def device_flags(self, clear: bool = False) -> int:
        """The MAPLE_FLAG_* bits that any layer's kernels have raised (synchronises)."""
        bits = 0
        for attn, moe in self.layers:
            bits |= int(attn.flags.item()) | moe.device_flags(clear)
            if clear:
                attn.flags.zero_()
        return bits
