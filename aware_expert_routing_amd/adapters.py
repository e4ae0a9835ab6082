"""Tables of low-rank adapters for one projection.

A table holds one stable handle per adapter in device memory; publishing,
replacing or clearing an adapter rewrites its handle on the stream (as expert
versions are published), so a captured graph that reads the table follows it.
"""
from __future__ import annotations

import torch

from . import _lib as L


class LoraTable:
    """n adapters of a projection [O, H], each of rank at most max_rank, none
    published yet (the table is cleared on the current stream; another stream
    that publishes into it or reads it has to come after that)."""

    def __init__(self, n: int, H: int, O: int, max_rank: int, device="cuda"):
        if n < 1:
            raise ValueError("a table holds at least one adapter")
        if not 1 <= max_rank <= 256:
            raise ValueError("max_rank must be in [1, 256]")
        if H < 32 or H % 32 or O < 16 or O % 16:
            raise ValueError("H must be a positive multiple of 32 and O of 16")
        self.n, self.H, self.O = n, H, O
        self.max_rank = (max_rank + 15) // 16 * 16
        self.handles = torch.zeros(n * L.LORA_HANDLE_BYTES, dtype=torch.uint8, device=torch.device(device))
        self._kept: dict[int, tuple] = {}   # the packed matrices each published handle points at

    def publish(self, i: int, a: torch.Tensor, b: torch.Tensor, scale: float = 1.0, stream=None):
        """Pack A [rank, H] and B [O, rank] (bf16) and make them adapter i
        (ordered on the stream).  The previous version's memory is released
        to the allocator: work on other streams that may still read it must
        be waited for first."""
        if not 0 <= i < self.n:
            raise ValueError(f"adapter {i} is outside the table")
        if a.dim() != 2 or b.dim() != 2 or a.shape[1] != self.H or b.shape[0] != self.O or a.shape[0] != b.shape[1]:
            raise ValueError(f"A must be [rank, {self.H}] and B [{self.O}, rank]")
        if not 1 <= a.shape[0] <= self.max_rank:
            raise ValueError(f"rank {a.shape[0]} is outside [1, {self.max_rank}]")
        pa, pb, rank = L.lora_pack(a, b, stream)
        h = L.LoraHandle()
        h.rank, h.scale, h.a, h.b, h.reserved = rank, scale, pa.data_ptr(), pb.data_ptr(), 0
        L.lora_publish(self.handles, i, h, stream)
        self._kept[i] = (pa, pb)

    def clear(self, i: int, stream=None):
        """Adapter i adds nothing from here on (ordered on the stream)."""
        L.lora_publish(self.handles, i, L.LoraHandle(), stream)
        self._kept.pop(i, None)
