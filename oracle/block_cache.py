"""Oracle for the block-scaled 8-bit cache: quantising blocks of 16 tokens and
one head, the prologue that writes them and the values they stand for.

TEST INFRASTRUCTURE ONLY: the tests may use this module; the product path
never does.

For one head, K and V apart, the tokens that one call writes into one block
(a run) are quantised with one scale: s* is the smallest power of two >= 2^-126
with max |y| <= 448 s* over the run's finite values; a run that holds the
block's first position sets s = s*, any other s = max(s_old, s*) and brings the
block's other codes to the new scale; the codes are E4M3(y / s).  fp64 numpy.
"""

from __future__ import annotations

import numpy as np

from . import rope_norm as rn

BLOCK = 16


def pow2_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def run_scale(y, old: float | None) -> float:
    """Scale of a block after a run of rows y; old None: the run starts it."""
    mag = np.abs(np.asarray(y, dtype=np.float64))
    mag = mag[np.isfinite(mag)]
    s = pow2_scale(float(mag.max()) if mag.size else 0.0)
    if old is None or not (np.isfinite(old) and old > 0):
        return s
    return max(float(old), s)


def values(codes, kv_scale, which: int) -> np.ndarray:
    """fp64 [P, 64, Hkv, D] that codes [P, 64, Hkv, D] stand for; kv_scale
    [P, Hkv, 2, 4], which 0: K, 1: V."""
    s = np.repeat(np.asarray(kv_scale, dtype=np.float64)[:, :, which], BLOCK, axis=2)
    return rn.e4m3_decode(codes) * s.transpose(0, 2, 1)[..., None]


def quantise_pages(x):
    """(codes, scales [P, Hkv, 4]) of whole pages x fp64 [P, 64, Hkv, D]."""
    P, page, Hkv, D = x.shape
    codes = np.zeros(x.shape, dtype=np.uint8)
    scales = np.zeros((P, Hkv, page // BLOCK))
    for p in range(P):
        for h in range(Hkv):
            for b in range(page // BLOCK):
                y = x[p, b * BLOCK:(b + 1) * BLOCK, h]
                s = run_scale(y, None)
                scales[p, h, b] = s
                codes[p, b * BLOCK:(b + 1) * BLOCK, h] = rn.e4m3_encode(y / s)
    return codes, scales


def write(rows, positions, token_req, block_table, codes, scales, page: int = 64):
    """Writes rows fp64 [N, Hkv, D] (one of K, V) into copies of codes [P, page,
    Hkv, D] and scales [P, Hkv, 4]; returns (codes, scales, runs, flags), runs as
    [(page, block, token indices)]."""
    codes, scales = np.array(codes, copy=True), np.array(scales, dtype=np.float64, copy=True)
    B, max_pages = block_table.shape
    flags, runs, prev = 0, [], None
    for t, pos in enumerate(positions):
        pos = int(pos)
        r = t if token_req is None else int(token_req[t])
        key = None
        if not (0 <= r < B and 0 <= pos < max_pages * page):
            flags |= 1
        elif not 0 <= int(block_table[r, pos // page]) < codes.shape[0]:
            flags |= 4
        else:
            key = (r, pos // BLOCK)
        if key is not None and key == prev:
            if len(runs[-1][2]) < BLOCK:
                runs[-1][2].append(t)
            else:
                flags |= 1
        elif key is not None:
            runs.append((int(block_table[r, pos // page]), pos % page // BLOCK, [t]))
        prev = key
    for pg, b, toks in runs:
        offs = [int(positions[t]) % BLOCK for t in toks]
        fresh = 0 in offs
        for h in range(codes.shape[2]):
            old = None if fresh else float(scales[pg, h, b])
            s = run_scale(rows[toks, h], old)
            blk = codes[pg, b * BLOCK:(b + 1) * BLOCK, h]
            if not fresh and s != old:
                keep = old if np.isfinite(old) and old > 0 else 0.0
                for o in set(range(BLOCK)) - set(offs):
                    blk[o] = rn.e4m3_encode(rn.e4m3_decode(blk[o]) * (keep / s))
            for t, o in zip(toks, offs):
                blk[o] = rn.e4m3_encode(rows[t, h] / s)
            scales[pg, h, b] = s
    return codes, scales, runs, flags
