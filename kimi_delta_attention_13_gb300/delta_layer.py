"""A layer of the gated delta rule with one decay per head, for prompts and single tokens.

Beside `linear_layer.LinearLayer`, whose frame it shares (residual norm in front, head norm, gate and
output projection behind), with the delta rule as its mixer and queries and keys shared by value heads:

    x, h     = residual_norm(x, y)                 add the block before, this block's input norm
    q, k, v, z, a, b = projections of h            q and k of unit norm
    g, beta  = -softplus(a + bias), sigmoid(b)     log decay and write gate per token and value head
    o        = delta_prefill / delta_decode        the recurrence, fp32 state carried
    y        = (norm_gate(o, z)) W_o               head norm and gate, output projection

The states are [N, H, d_k, d_v] fp32, as the KDA layers' own, so that `prefix_cache.CheckpointStore`
holds them too, as they are or in fewer bits.  `delta_prefill` emits no checkpoints on its way: what can be stored is
the state at a call's end, sequence i's by `store.add_checkpoints([key], state[i:i + 1], n, [n])` at its length n (or by
`store.write`); a prompt that continues it takes `store.read`'s states as `prefill`'s `state` (`resume_prefill` is for
the KDA layers).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import delta_decode, delta_prefill, residual_norm
from .linear_layer import LinearLayer


class DeltaLayer(LinearLayer):
    """Random-initialised weights of one layer; `prefill` runs packed prompts, `decode` one token per
    sequence from the states that `prefill` left.  `heads` value heads share `key_heads` heads of queries
    and keys."""

    def __init__(self, width: int, heads: int, key_heads: Optional[int] = None, d_k: int = 128, d_v: int = 128, *,
                 residual_scale: float = 1.0, eps: float = 1e-6, device="cuda", dtype=torch.bfloat16, seed: int = 0):
        key_heads = heads if key_heads is None else key_heads
        if key_heads < 1 or heads % key_heads != 0:
            raise ValueError(f"{heads} value heads cannot share {key_heads} query/key heads evenly")
        self.heads, self.key_heads, self.d_k, self.d_v = heads, key_heads, d_k, d_v
        self.scale, self.residual_scale, self.eps, self.dtype = d_k ** -0.5, residual_scale, eps, dtype
        gen = torch.Generator(device=device).manual_seed(seed)
        self._split = [key_heads * d_k, key_heads * d_k, heads * d_v, heads * d_v, heads, heads]
        normal = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
        self.w_in = (normal(width, sum(self._split)) * width ** -0.5).to(dtype)
        self.w_out = (normal(heads * d_v, width) * (heads * d_v) ** -0.5).to(dtype)
        self.bias = normal(heads) - 3.0                 # decays of some 4 to 200 tokens' memory
        self.n_in, self.n_post = torch.ones(width, device=device), torch.ones(width, device=device)
        self.n_head = torch.ones(d_v, device=device)

    def _enter(self, x: torch.Tensor, y: Optional[torch.Tensor]):
        """The residual stream after the block before, and the mixer's operands."""
        post = None if y is None else self.n_post
        x, h = residual_norm(x, y, self.n_in, w_post=post, scale=self.residual_scale, eps=self.eps,
                             out_dtype=self.dtype)
        q, k, v, z, a, b = (h @ self.w_in).split(self._split, dim=1)
        rows = x.shape[0]
        q, k = (torch.nn.functional.normalize(t.reshape(rows, self.key_heads, self.d_k), dim=-1) for t in (q, k))
        v, z = (t.reshape(rows, self.heads, self.d_v).contiguous() for t in (v, z))
        g = -torch.nn.functional.softplus(a.float() + self.bias)
        return x, (q, k, v, g, torch.sigmoid(b.float())), z

    def prefill(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                state: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """Packed prompts x [T, width] (the residual stream) and the block before's output y [T, width]
        (None for a first block).  Returns (residual stream, this block's output, states)."""
        x, mixer, z = self._enter(x, y)
        o, state = delta_prefill(*mixer, cu_seqlens, state, scale=self.scale)
        return x, self._leave(o, z), state

    def decode(self, x: torch.Tensor, y: Optional[torch.Tensor], state: torch.Tensor) \
            -> Tuple[torch.Tensor, torch.Tensor]:
        """One token per sequence, x and y [N, width]; `state` is updated in place.  Returns (residual
        stream, this block's output)."""
        x, mixer, z = self._enter(x, y)
        return x, self._leave(delta_decode(*mixer, state, scale=self.scale), z)
