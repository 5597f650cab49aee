"""CPU oracle of the attention over a key/value cache and of its eviction.

TEST INFRASTRUCTURE ONLY, like ``area_oracle``: plain NumPy in float64 from the
definitions in include/area.h, sharing no code with the library.
"""
from __future__ import annotations

from typing import Optional

import numpy as np


def visible(n: int, Nq: int, S: int, window: Optional[int] = None, sinks: int = 0,
            causal: bool = True) -> np.ndarray:
    """[Nq, S] truth values: the tokens of an n-token sequence that each of its
    last Nq queries sees (query i sits at position n - Nq + i)."""
    p = n - Nq + np.arange(Nq)[:, None]
    j = np.arange(S)[None, :]
    if not causal:
        return np.broadcast_to(j < n, (Nq, S))
    see = j <= p
    if window is not None:
        see = see & ((j > p - window) | (j < sinks))
    return see


def masked_attention(q, k, v, see, scale):
    """One head.  q [Nq, D], k, v [n, D], see [Nq, n] -> output [Nq, D], weights
    [Nq, n], the sum of weight times |value| [Nq, D].  Only what is seen is
    used; a query that sees nothing has no weights and a row of zeros."""
    Nq = q.shape[0]
    q = np.asarray(q, np.float64)
    w = np.zeros(see.shape, np.float64)
    o = np.zeros((Nq, v.shape[1]), np.float64)
    size = np.zeros_like(o)
    for i in range(Nq):
        at = np.flatnonzero(see[i])
        if at.size == 0:
            continue
        x = scale * (np.asarray(k, np.float64)[at] @ q[i])
        e = np.exp(x - x.max())
        w[i, at] = e / e.sum()
        vals = np.asarray(v, np.float64)[at]
        o[i] = w[i, at] @ vals
        size[i] = w[i, at] @ np.abs(vals)
    return o, w, size


def cache_attention(q, k, v, lens, scale, window=None, sinks=0, causal=True, kp=None, vp=None):
    """q [B, H, Nq, D]; k, v [B, Hk, S, D]; kp, vp [Hk, P, D] or None.  Returns
    the output, the weights that each own key got from its key head's rows
    [B, Hk, S], and the sum of weight times |value| per output."""
    B, H, Nq, D = q.shape
    Hk, S = k.shape[1], k.shape[2]
    o, size = np.zeros((B, H, Nq, D)), np.zeros((B, H, Nq, D))
    got = np.zeros((B, Hk, S))
    P = 0 if kp is None else kp.shape[1]
    for b in range(B):
        n = min(max(int(lens[b]), 0), S)
        mine = visible(n, Nq, S, window, sinks, causal)
        before = np.ones((Nq, P), bool)
        if causal:
            before &= (n - Nq + np.arange(Nq) >= 0)[:, None]
        see = np.concatenate([before, mine], 1)
        for h in range(H):
            hk = h // (H // Hk)
            kk, vv = k[b, hk], v[b, hk]
            if P:
                kk, vv = np.concatenate([kp[hk], kk]), np.concatenate([vp[hk], vv])
            o[b, h], w, size[b, h] = masked_attention(q[b, h], kk, vv, see, scale)
            got[b, hk] += w[:, P:].sum(0)
    return o, got, size


def kept_tokens(acc, n: int, budget: int, sinks: int, recent: int) -> list:
    """Positions that one key head keeps of its n tokens (acc [>= n])."""
    if n <= budget:
        return list(range(n))

    def heaviest_first(j):
        w = float(acc[j])
        return (-(float("-inf") if w != w else w), j)

    free = sorted(range(sinks, n - recent), key=heaviest_first)
    return sorted(list(range(sinks)) + free[:budget - sinks - recent]
                  + list(range(n - recent, n)))
