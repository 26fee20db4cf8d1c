"""Oracle for windowed attention with sinks, over any paged cache.

TEST INFRASTRUCTURE ONLY: the tests may use this module; the product path
never does.

A query at position p of its request sees token j <= p when j > p - window or
j < sinks (window = 0: every token up to p).  The request's last q_len tokens
are the queries.  A query that sees nothing yields a zero row.  Everything is
fp64 numpy, one request and query head at a time.
"""

from __future__ import annotations

import numpy as np


def visible(L: int, q_len: int, window: int, sinks: int) -> np.ndarray:
    """bool [q_len, L]: token j is seen by query i (position L - q_len + i)."""
    p = L - q_len + np.arange(q_len)[:, None]
    j = np.arange(L)[None, :]
    see = (j <= p) & (p >= 0)
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def gather(pages, table, L: int, page: int = 64) -> np.ndarray:
    """Rows 0 .. L - 1 of a request from fp64 pages [P, page, Hkv, D]; a page no
    valid entry names is NaN (it must not be looked at)."""
    n = -(-L // page)
    out = np.full((n * page,) + pages.shape[2:], np.nan)
    for t in range(n):
        g = int(table[t])
        if 0 <= g < pages.shape[0]:
            out[t * page:(t + 1) * page] = pages[g]
    return out[:L]


def attention(q, k_pages, v_pages, block_table, seqlens, window: int, sinks: int, sm_scale: float):
    """(out, mass) fp64 [B, q_len, Hq, D]: the attention and sum_j w_j |v_j|, the
    size its weights' rounding errors act on.  q fp64 [B, q_len, Hq, D];
    k_pages, v_pages fp64 [P, page, Hkv, D]."""
    B, n, Hq, D = q.shape
    G = Hq // k_pages.shape[2]
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    for r in range(B):
        L = int(seqlens[r])
        if L <= 0:
            continue
        see = visible(L, n, window, sinks)
        some = see.any(0)  # tokens nobody sees are left out, whatever they hold
        K = gather(k_pages, block_table[r], L)[some]
        V = gather(v_pages, block_table[r], L)[some]
        mask = see[:, some]
        for h in range(Hq):
            x = q[r, :, h] @ K[:, h // G].T * sm_scale
            x = np.where(mask, x, -np.inf)
            m = x.max(-1, keepdims=True, initial=-np.inf)
            e = np.exp(x - np.where(np.isfinite(m), m, 0.0))
            z = e.sum(-1, keepdims=True)
            w = np.divide(e, z, out=np.zeros_like(e), where=z > 0)
            out[r, :, h] = w @ V[:, h // G]
            mass[r, :, h] = w @ np.abs(V[:, h // G])
    return out, mass


def planned_lengths(seqlens, max_pages: int, q_len: int, window: int, sinks: int,
                    page: int = 64) -> list:
    """Lengths whose tiles a windowed plan cuts: each request without the tiles
    that lie behind its sinks and before its first query's window."""
    out = []
    for L in seqlens:
        L = min(max(int(L), 0), page * max_pages)
        tiles = -(-L // page)
        if window and L:
            lo = max(0, L - q_len + 1 - window)
            kept = sum(1 for t in range(tiles) if t < -(-sinks // page) or t >= lo // page)
            L -= page * (tiles - kept)
        out.append(L)
    return out
