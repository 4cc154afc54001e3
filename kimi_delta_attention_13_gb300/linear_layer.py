"""A linear-attention layer for prompts and single tokens, from the library's calls.

The block around a mixer whose heads each have one decay, as a hybrid model stacks it between its
KDA layers:

    x, h  = residual_norm(x, y)             add the block before (its post-norm and residual scale),
                                            then this block's input norm
    q, k, v, z, a = projections of h        (library matrix products)
    g     = -softplus(a + bias)             log decay per token and head
    o     = linear_prefill / linear_decode  the recurrence, fp32 state carried
    y     = (norm_gate(o, z)) W_o           head norm and gate, output projection

The states are [N, H, d_k, d_v] fp32, as the KDA layers' own, so that `state_copy` and
`prefix_cache.CheckpointStore` hold and restore them too (a prompt's final state as one checkpoint, at
the prompt's length).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import linear_decode, linear_prefill, norm_gate, residual_norm


class LinearLayer:
    """Random-initialised weights of one layer; `prefill` runs packed prompts, `decode` one token per
    sequence from the states that `prefill` left.  The residual stream may be bf16 or fp32, whatever the
    layer's dtype; block outputs have the layer's."""

    def __init__(self, width: int, heads: int, kv_heads: Optional[int] = None, d_k: int = 128, d_v: int = 128, *,
                 residual_scale: float = 1.0, eps: float = 1e-6, device="cuda", dtype=torch.bfloat16, seed: int = 0):
        kv_heads = heads if kv_heads is None else kv_heads
        if kv_heads < 1 or heads % kv_heads != 0:
            raise ValueError(f"{heads} query heads cannot share {kv_heads} key/value heads evenly")
        self.heads, self.kv_heads, self.d_k, self.d_v = heads, kv_heads, d_k, d_v
        self.scale, self.residual_scale, self.eps, self.dtype = d_k ** -0.5, residual_scale, eps, dtype
        gen = torch.Generator(device=device).manual_seed(seed)
        self._split = [heads * d_k, kv_heads * d_k, kv_heads * d_v, heads * d_v, heads]
        normal = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
        self.w_in = (normal(width, sum(self._split)) * width ** -0.5).to(dtype)
        self.w_out = (normal(heads * d_v, width) * (heads * d_v) ** -0.5).to(dtype)
        self.bias = normal(heads) - 3.0                 # decays of some 4 to 200 tokens' memory
        self.n_in, self.n_post = torch.ones(width, device=device), torch.ones(width, device=device)
        self.n_head = torch.ones(d_v, device=device)

    def _enter(self, x: torch.Tensor, y: Optional[torch.Tensor]):
        """The residual stream after the block before, and this block's operands."""
        post = None if y is None else self.n_post
        x, h = residual_norm(x, y, self.n_in, w_post=post, scale=self.residual_scale, eps=self.eps,
                             out_dtype=self.dtype)
        q, k, v, z, a = (h @ self.w_in).split(self._split, dim=1)
        rows = x.shape[0]
        q = q.reshape(rows, self.heads, self.d_k).contiguous()
        k = torch.nn.functional.normalize(k.reshape(rows, self.kv_heads, self.d_k), dim=-1)
        v = v.reshape(rows, self.kv_heads, self.d_v).contiguous()
        z = z.reshape(rows, self.heads, self.d_v).contiguous()
        g = -torch.nn.functional.softplus(a.float() + self.bias)
        return x, q, k, v, z, g

    def _leave(self, o: torch.Tensor, z: torch.Tensor) -> torch.Tensor:
        return norm_gate(o, z, self.n_head, eps=self.eps, out=o).flatten(1) @ self.w_out

    def prefill(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                state: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """Packed prompts x [T, width] (the residual stream) and the block before's output y [T, width]
        (None for a first block).  Returns (residual stream, this block's output, states)."""
        x, q, k, v, z, g = self._enter(x, y)
        o, state = linear_prefill(q, k, v, g, cu_seqlens, state, scale=self.scale)
        return x, self._leave(o, z), state

    def decode(self, x: torch.Tensor, y: Optional[torch.Tensor], state: torch.Tensor) \
            -> Tuple[torch.Tensor, torch.Tensor]:
        """One token per sequence, x and y [N, width]; `state` is updated in place.  Returns (residual
        stream, this block's output)."""
        x, q, k, v, z, g = self._enter(x, y)
        return x, self._leave(linear_decode(q, k, v, g, state, scale=self.scale), z)
