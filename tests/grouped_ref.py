"""Grouped routing by its definition in 64 bits, token by token (numpy), and
the dispatch lists of a routing result."""
from __future__ import annotations

import numpy as np


def route_grouped(logits, k, score, bias, n_group, topk_group, group_score, renorm, scale, n_valid=None):
    """logits [B, N] float32 values.  Returns (idx int32 [B, k], w float64 [B, k])."""
    B, N = logits.shape
    per = N // n_group
    idx = np.full((B, k), -1, np.int32)
    w = np.zeros((B, k))
    for i in range(B if n_valid is None else min(max(n_valid, 0), B)):
        l = np.minimum(logits[i].astype(np.float64), float(np.finfo(np.float32).max))
        live = l > -np.inf   # False for NaN
        if not live.any():
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                s = np.where(live, np.exp(np.where(live, l, 0.0) - l[live].max()), 0.0)
                s = s / s.sum()
            else:
                s = np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, l, 0.0))), 0.0)
        c = l.copy() if bias is None else s + bias.astype(np.float64)
        c[~live | ~(c > -np.inf)] = -np.inf
        if n_group > 1:
            by_sum = group_score == "top2" and per > 1
            value = np.full(n_group, -np.inf)
            for g in range(n_group):
                at = slice(g * per, (g + 1) * per)
                ok = c[at] > -np.inf
                if not ok.any():
                    continue
                v = np.sort((s if bias is None and by_sum else c)[at][ok])[::-1]
                value[g] = v[:2].sum() if by_sum else v[0]
            order = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            for g in range(n_group):
                if g not in order or value[g] == -np.inf:
                    c[g * per:(g + 1) * per] = -np.inf
        pick = [e for e in sorted(range(N), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:k]
        p = s[pick]
        if renorm:
            p = p / p.sum() if p.sum() > 0 else p * 0.0
        idx[i, :len(pick)] = pick
        w[i, :len(pick)] = p * scale
    return idx, w


def dispatch(idx, N):
    B, k = idx.shape
    pairs = sorted((int(e), q) for q, e in enumerate(idx.reshape(-1)) if 0 <= e < N)
    cnt = np.zeros(N, np.int32)
    for e, _ in pairs:
        cnt[e] += 1
    perm = np.full(B * k, -1, np.int32)
    perm[:len(pairs)] = [q for _, q in pairs]
    active = np.full(N, -1, np.int32)
    on = np.nonzero(cnt)[0]
    active[:len(on)] = on
    return dict(cnt=cnt, offsets=np.concatenate([[0], np.cumsum(cnt)]).astype(np.int32), perm=perm, active=active,
                T=np.array([len(on)], np.int32))
