"""The oracle of the page pool against what has to hold of any pool."""

import random

import pytest

from oracle import pages as op


def consistent(pool):
    named = [p for row in pool["table"] for p in row if p >= 0]
    assert pool["refs"] == [named.count(p) for p in range(len(pool["refs"]))]
    assert sorted(pool["stack"]) == [p for p, r in enumerate(pool["refs"]) if r == 0]


@pytest.mark.parametrize("seed", range(20))
def test_any_sequence_leaves_every_page_held_or_free(seed):
    r = random.Random(seed)
    pool = op.new(8, 10, 50)
    lens = [0] * 8
    for _ in range(60):
        what = r.choice(["extend", "free", "fork", "compact"])
        if what == "extend":
            rows = r.sample(range(8), r.randint(0, 8))
            want = [r.randint(lens[b], 640) for b in rows]
            if op.extend(pool, rows, want):
                for b, L in zip(rows, want):
                    lens[b] = L
        elif what == "free":
            rows = r.sample(range(8), r.randint(0, 4))
            keep = [r.randint(0, lens[b]) for b in rows]
            op.free(pool, rows, keep)
            for b, L in zip(rows, keep):
                lens[b] = L
        elif what == "fork":
            empty = [b for b in range(8) if lens[b] == 0]
            full = [b for b in range(8) if lens[b] > 0]
            if full:
                src = [r.choice(full) for _ in empty]
                cut = [r.randint(0, lens[a]) for a in src]
                if op.fork(pool, src, empty, cut) is not None:
                    for b, L in zip(empty, cut):
                        lens[b] = L
        else:
            op.compact(pool)
            live = sum(n > 0 for n in pool["refs"])
            assert all(n > 0 for n in pool["refs"][:live])
        consistent(pool)
        assert all(sum(p >= 0 for p in row) == op.pages_of(L)
                   for row, L in zip(pool["table"], lens))


def test_freed_rows_get_their_pages_again():
    pool = op.new(4, 8, 20)
    op.extend(pool, [2, 0], [300, 100])
    before = [list(r) for r in pool["table"]]
    op.free(pool, [2, 0])
    op.extend(pool, [2, 0], [300, 100])
    assert pool["table"] == before
