"""A projection with adapters and the shared expert in 64 bits (torch, on the
CPU), with the magnitudes that the tests' error bounds use."""
from __future__ import annotations

import torch


def make_table(seed: int, n: int, H: int, O: int, ranks, empty=()):
    """n adapters (A [r, H], B [O, r] bf16 on the CPU, scale); None where empty."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for a in range(n):
        r = ranks[a % len(ranks)]
        A = (torch.randn(r, H, generator=g) * H ** -0.5).to(torch.bfloat16)
        B = (torch.randn(O, r, generator=g) * 0.3).to(torch.bfloat16)
        out.append(None if a in empty else (A, B, 0.25 + 0.25 * (a % 5)))
    return out


def linear(x, W, table, ids):
    """x [B, H] float64 through W and the adapters.  Returns (y, sum |W||x|,
    sum over the adapter of s |B| (|A| |x|))."""
    W = W.double()
    y, mag, lmag = x @ W.T, x.abs() @ W.abs().T, torch.zeros(x.shape[0], W.shape[0], dtype=torch.float64)
    for a, entry in enumerate(table or []):
        at = (ids == a).nonzero().flatten()
        if entry is None or at.numel() == 0:
            continue
        A, B, s = entry
        y[at] += s * (x[at] @ A.double().T) @ B.double().T
        lmag[at] += s * (x[at].abs() @ A.double().abs().T) @ B.double().abs().T
    return y, mag, lmag


def shared(x, gate, up, down, tables, ids):
    g, u = linear(x, gate, tables[0], ids)[0], linear(x, up, tables[1], ids)[0]
    return linear(g * torch.sigmoid(g) * u, down, tables[2], ids)[0]
