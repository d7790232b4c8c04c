"""Accumulated attention weights and eviction by them, in plain numpy and 64 bits.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with the CUDA path.
Pools are [pages, P, Hkv, D] (layout "nhd") or [pages, Hkv, P, D] ("hnd"), uint16 bit patterns.
"""
from __future__ import annotations

import math

import numpy as np

from .int4 import bf16_value


def _by_position(pool, layout):
    return pool if layout == "nhd" else pool.transpose(0, 2, 1, 3)


def weights(q, k_pool, block_table, context_lens, scale=None, layout="nhd") -> list:
    """Per sequence fp64 [Hkv, ctx]: the softmax weights summed over each kv head's query heads."""
    pool = _by_position(k_pool, layout)
    P, H, D = pool.shape[1:]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    out = []
    for s, n in enumerate(context_lens):
        p = np.arange(int(n))
        k = bf16_value(pool[block_table[s][p // P], p % P]).astype(np.float64)
        qs = bf16_value(q[s]).astype(np.float64).reshape(H, -1, D)
        x = np.einsum("hgd,lhd->hgl", qs, k) * scale
        if n:
            x = np.exp(x - x.max(-1, keepdims=True))
            x /= x.sum(-1, keepdims=True)
        out.append(x.sum(1))
    return out


def kept(w, pos, budget, recent, last=None) -> np.ndarray:
    """Which of a row's slots stay (weights w and original positions pos of its slots; last: the
    newest token's position, by default the last slot's)."""
    n = min(len(w), budget)
    stay = np.zeros(len(w), bool)
    if len(w) == 0:
        return stay
    newest = pos > (int(pos[-1]) if last is None else last) - recent
    w = np.where(np.isnan(w), -np.inf, w.astype(np.float64))
    order = sorted(range(len(w)), key=lambda i: (not newest[i], 0.0 if newest[i] else -w[i], i))
    stay[order[:n]] = True
    return stay


def evict(k_pool, v_pool, w, pos, block_table, context_lens, budget, recent, rows=None,
          layout="nhd", newest=None):
    """In place on the pools and on w, pos ([rows, Hkv, stride]); returns the new lengths.  newest[s]:
    the position of sequence s's newest token, by default that of its last slot (a sequence that has
    had no token since its last cut may hold any token there)."""
    kp, vp = _by_position(k_pool, layout), _by_position(v_pool, layout)
    P, H = kp.shape[1:3]
    new_lens = []
    for s, n_all in enumerate(context_lens):
        row = s if rows is None else int(rows[s])
        if row < 0:
            new_lens.append(int(n_all))
            continue
        n = min(int(n_all), budget)
        new_lens.append(n)
        for h in range(H):
            ww, pp = w[row, h], pos[row, h]
            last = -1 if n_all == 0 else int(pp[n_all - 1] if newest is None else newest[s])
            total = last + 1
            stay = kept(ww[:n_all], pp[:n_all], budget, recent, last)
            gaps = np.flatnonzero(~stay[:n])
            movers = n + np.flatnonzero(stay[n:])
            for g, m in zip(gaps, movers):
                to, at = (block_table[s][g // P], g % P, h), (block_table[s][m // P], m % P, h)
                kp[to], vp[to] = kp[at], vp[at]
                ww[g], pp[g] = ww[m], pp[m]
            ww[n:n_all] = 0.0
            pp[n:] = total + np.arange(len(pp) - n)
    return np.array(new_lens, dtype=np.int32)
