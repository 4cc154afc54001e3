"""Prefix reuse for KDA serving: resume a request from a stored state checkpoint.

Page "Kimi K3 im Detail: Delta Attention, Attention über Schichten und LatentMoE", section
"Sequenz-Mixing: KDA-Zustand und globale MLA": a reused prefix has to restart from the KDA state
at the same token boundary, and that state is stored only at sparse checkpoints. A request whose
first tokens match a cached sequence therefore:
1. restores the state of the longest checkpoint within the shared prefix (`kda_state_copy`);
2. prefills only the tokens after it, starting from that state (`kda_prefill` with `init_state`).

States may be kept in fewer bits than they are worked on in (`CheckpointStore(..., dtype=...)`): packed as
they are stored (`kda_state_pack`), read back as they are restored (`kda_state_unpack`).

`CheckpointStore` is a device pool of checkpoint slots with a host-side index. It takes the
checkpoints a prefill emitted (`ckpt_stride`, `ckpts`), and answers "which slot holds the state
after n tokens of sequence `key`". `resume_prefill` restores a batch of requests from their slots in
one `kda_state_copy` (or `kda_state_unpack`) and runs one varlen `kda_prefill` over their remaining tokens.

All device work goes through the library's C ABI; this module only keeps the index.
"""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import _on_stream, num_checkpoints, prefill, state_copy, state_pack, state_unpack


class CheckpointStore:
    """A pool of `n_slots` states [n_slots, H, d_k, d_v] on `device`, filled round-robin
    (the oldest entry is overwritten when the pool is full), indexed by (key, tokens covered).
    dtype: float32 (as they are), int8 (a quarter of the memory: a value is off by at most 1/254 of its
    row's largest, rows being key channels, whose scales are `scales`), or bfloat16 (half: at most 2^-8 of
    the value); packed ones have d_v a multiple of 4, d_k and d_v up to 256."""

    def __init__(self, n_slots: int, heads: int, d_k: int = 128, d_v: int = 128, device=None,
                 dtype: torch.dtype = torch.float32):
        if n_slots < 1:
            raise ValueError("n_slots must be positive")
        if dtype not in (torch.float32, torch.bfloat16, torch.int8):
            raise ValueError("a store holds float32, bfloat16 or int8 states")
        if dtype is not torch.float32 and (d_v % 4 != 0 or d_v > 256 or d_k > 256):   # kda_state_pack's
            raise ValueError(f"states of {d_k} x {d_v} cannot be packed: d_v a multiple of 4, both up to 256")
        self.states = torch.empty(n_slots, heads, d_k, d_v, device=device, dtype=dtype)
        self.scales = torch.empty(n_slots, heads, d_k, device=device) if dtype is torch.int8 else None
        self._index: Dict[Tuple[object, int], int] = {}
        self._owner: List[Optional[Tuple[object, int]]] = [None] * n_slots
        self._next = 0

    @property
    def n_slots(self) -> int:
        return self.states.shape[0]

    def write(self, slots: torch.Tensor, states: torch.Tensor, rows: torch.Tensor, stream=None) -> None:
        """states[rows[i]] into slot slots[i] (int64 device tensors, the slots all different)."""
        if self.states.dtype is torch.float32:
            state_copy(self.states, states, slots, rows, stream=stream)
        else:
            state_pack(self.states, states, slots, rows, scales=self.scales, stream=stream)

    def read(self, states: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """states[rows[i]] = what slot slots[i] holds, in fp32."""
        if self.states.dtype is torch.float32:
            state_copy(states, self.states, rows, slots, stream=stream)
        else:
            state_unpack(states, self.states, rows, slots, scales=self.scales, stream=stream)

    def _take_slot(self, entry: Tuple[object, int]) -> int:
        slot = self._next
        self._next = (self._next + 1) % self.n_slots
        old = self._owner[slot]
        if old is not None and self._index.get(old) == slot:
            del self._index[old]
        prev = self._index.get(entry)
        if prev is not None:   # the same checkpoint stored again: its older slot is superseded
            self._owner[prev] = None
        self._owner[slot] = entry
        self._index[entry] = slot
        return slot

    def add_checkpoints(self, keys: Sequence[object], ckpts: torch.Tensor, ckpt_stride: int,
                        lengths: Sequence[int], stream=None) -> List[Tuple[object, int, int]]:
        """Store the checkpoints a prefill of sequences `lengths` emitted with `ckpt_stride`
        (`ckpts` as returned by `prefill`, slots ordered by sequence then position), under the
        sequences' `keys`. Returns (key, tokens covered, slot) per stored checkpoint."""
        if len(keys) != len(lengths):
            raise ValueError("one key per sequence")
        if ckpts.shape[0] != num_checkpoints(lengths, ckpt_stride):
            raise ValueError("ckpts does not match lengths and ckpt_stride")
        entries, src = [], []
        pos = 0
        for key, n in zip(keys, lengths):
            for m in range(1, n // ckpt_stride + 1):
                entries.append((key, m * ckpt_stride))
                src.append(pos)
                pos += 1
        if len(entries) > self.n_slots:
            raise ValueError(f"{len(entries)} checkpoints do not fit {self.n_slots} slots")
        dst = [(self._next + i) % self.n_slots for i in range(len(entries))]
        if entries:
            dev = self.states.device
            with _on_stream(dev, stream):   # what the copy reads belongs to its stream
                slots, rows = (torch.tensor(x, device=dev, dtype=torch.int64) for x in (dst, src))
            self.write(slots, ckpts, rows, stream=stream)
        for e in entries:                   # indexed once they are written: a refused copy leaves the store as it was
            self._take_slot(e)
        return [(k, n, s) for (k, n), s in zip(entries, dst)]

    def lookup(self, key: object, n_tokens: int) -> Tuple[Optional[int], int]:
        """The slot holding the state after the most tokens of `key`, at most `n_tokens`, and that
        token count; (None, 0) if no checkpoint of `key` lies within the first `n_tokens`."""
        best = (None, 0)
        for (k, covered), slot in self._index.items():
            if k == key and covered <= n_tokens and covered > best[1]:
                best = (slot, covered)
        return best


def resume_prefill(store: CheckpointStore, slots: Sequence[Optional[int]], q, k, v, g, beta,
                   cu_seqlens: torch.Tensor, lengths: Sequence[int], *, out=None,
                   final_state=True, out_dtype=torch.float32, stream=None):
    """Prefill a batch of requests from restored states: request i continues from the state in
    `store` slot `slots[i]` (None: from zeros) over its remaining tokens, packed varlen in q, k,
    v, g, beta with `cu_seqlens` / `lengths`. Returns (out, final_state, init_states)."""
    n = len(lengths)
    if len(slots) != n:
        raise ValueError("one slot per request")
    _, H, dk, dv = store.states.shape
    dev = store.states.device
    pairs = [(i, s) for i, s in enumerate(slots) if s is not None]
    with _on_stream(dev, stream):   # zeros before the restored states, on their stream
        init = torch.zeros(n, H, dk, dv, device=dev, dtype=torch.float32)
        to, of = (torch.tensor([p[x] for p in pairs], device=dev, dtype=torch.int64) for x in (0, 1))
    if pairs:
        store.read(init, to, of, stream=stream)
    o, f, _ = prefill(q, k, v, g, beta, cu_seqlens, init, out=out, final_state=final_state,
                      lengths=lengths, out_dtype=out_dtype, stream=stream)
    return o, f, init
