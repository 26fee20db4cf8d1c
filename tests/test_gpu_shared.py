"""Decode attention over shared prefixes against the fp64 oracle."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from _shared import Shared

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "block"]
# (Hq, Hkv, q_len): query rows per KV head and request on both sides of 8, groups of heads
# that do not divide 128, odd and even numbers of KV heads
HEADS = [(8, 1, 1), (2, 2, 1), (16, 1, 1), (6, 2, 2), (3, 1, 5), (15, 3, 3), (16, 4, 3),
         (1, 1, 1), (12, 6, 8), (32, 2, 1), (5, 1, 1)]


def wide(n, pages, q_len, seed):
    """A group of n requests behind `pages` shared ones: some end at once, some tails fill
    tiles, two members are too short to share, one is empty."""
    r = np.random.default_rng(seed)
    lens = [64 * pages + q_len - 1 + int(t) for t in r.integers(0, 150, n)]
    lens[0] = 64 * pages + q_len - 1  # nothing behind the pages but the last queries
    if n > 5:
        lens[1], lens[3], lens[n - 1] = 64 * pages + q_len - 2, 0, 10
        lens[4] = 64 * pages + 64
    return lens


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("heads", range(len(HEADS)))
def test_one_group(kv, heads):
    hq, hkv, n = HEADS[heads]
    lens = wide(20, 3, n, heads)
    c = Shared(kv, lens, [0, 20], [3], hq, hkv, n, seed=500 + heads).to_gpu()
    for ctas in (2, 7, 0):
        got, ws = c.step(ctas=ctas)
        c.check_plan(ws)
        c.check(got)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("heads", [0, 3, 5, 6])
def test_several_groups(kv, heads):
    """Groups of one, of two, of many and of none that shares, requests of no group on
    both sides, no shared pages."""
    hq, hkv, n = HEADS[heads]
    lens = [300] + wide(1, 2, n, 1) + wide(2, 5, n, 2) + wide(33, 9, n, 3) + wide(7, 1, n, 4) + \
        [50, 700] + [40, 0, 30] + [500, 0, 129]
    starts, pages = [1, 2, 4, 37, 44, 46, 49], [2, 5, 9, 1, 0, 3]
    c = Shared(kv, lens, starts, pages, hq, hkv, n, seed=600 + heads).to_gpu()
    for ctas, floor in ((3, 0), (40, 2), (0, 2), (0, 9)):
        got, ws = c.step(ctas=ctas, floor=floor)
        c.check_plan(ws)
        c.check(got)


@pytest.mark.parametrize("kv", KINDS)
def test_row_tiles_in_pairs_and_alone(kv):
    """One, two, three and five row tiles of 128 rows; pages split between CTAs."""
    for B in (16, 17, 32, 48, 80):
        lens = wide(B, 4, 1, B)
        c = Shared(kv, lens, [0, B], [4], 8, 1, 1, seed=B).to_gpu()
        for ctas in (4, 0):
            got, ws = c.step(ctas=ctas)
            c.check_plan(ws)
            c.check(got)


@pytest.mark.parametrize("kv", KINDS)
def test_long_prefixes(kv):
    """Many pages per descriptor: the rings go round, the reference moves."""
    lens = wide(9, 150, 1, 5)
    c = Shared(kv, lens, [0, 9], [150], 16, 2, 1, seed=77).to_gpu()
    for ctas in (2, 5, 0):
        got, ws = c.step(ctas=ctas)
        c.check_plan(ws)
        c.check(got)
    lens = wide(36, 61, 1, 6)
    c = Shared(kv, lens, [0, 36], [61], 8, 1, 1, seed=78).to_gpu()
    for ctas in (2, 3, 0):
        got, _ = c.step(ctas=ctas)
        c.check(got)
