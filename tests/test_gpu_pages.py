"""The page pool on the GPU against its oracle: every result exactly."""

import random

import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as E
from oracle import pages as op

pytestmark = pytest.mark.gpu

IDLE = 2 ** 31 - 1


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool and a table on the device, and the oracle's."""

    def __init__(self, B, max_pages, num_pages):
        self.want = op.new(B, max_pages, num_pages)
        self.pool = hd.PagePool(num_pages)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.copies = torch.zeros((num_pages + B + 1, 2), dtype=torch.int32, device="cuda")

    def check(self, flags=0, copies=None):
        assert self.table.tolist() == self.want["table"]
        assert self.pool.refs.tolist() == self.want["refs"]
        n = len(self.want["stack"])
        assert self.pool.state.tolist() == [n, flags, 0, 0]
        assert self.pool.free_list[:n].tolist() == self.want["stack"]
        assert (self.pool.marks == IDLE).all()
        if copies is not None:
            assert self.copies[0].tolist() == [len(copies), 0]
            assert [tuple(c) for c in self.copies[1:1 + len(copies)].tolist()] == copies


def play(both, r, steps, check_each=True):
    """A sequence of calls on both."""
    B, cols = both.table.shape
    lens = [0] * B
    flags = 0
    for _ in range(steps):
        what = r.choice(["extend", "extend", "free", "fork", "compact"])
        copies = None
        if what == "extend":
            rows = r.sample(range(B), r.randint(0, B))
            want = [r.randint(lens[b], 64 * cols) for b in rows]
            hd.hpc_kv_extend(both.pool, both.table, ints(rows), ints(want))
            if op.extend(both.want, rows, want):
                for b, L in zip(rows, want):
                    lens[b] = L
            else:
                flags = E.HPC_FLAG_NO_PAGES
        elif what == "free":
            rows = r.sample(range(B), r.randint(0, B))
            keep = [r.randint(0, lens[b]) if r.random() < 0.5 else 0 for b in rows]
            hd.hpc_kv_free(both.pool, both.table, ints(rows), ints(keep))
            op.free(both.want, rows, keep)
            for b, L in zip(rows, keep):
                lens[b] = L
        elif what == "fork":
            full = [b for b in range(B) if lens[b] > 0]
            dst = [b for b in range(B) if lens[b] == 0]
            if not full:
                continue
            src = [r.choice(full) for _ in dst]
            cut = [r.randint(0, lens[a]) for a in src]
            hd.hpc_kv_fork(both.pool, both.table, ints(src), ints(dst), ints(cut), both.copies)
            copies = op.fork(both.want, src, dst, cut)
            if copies is None:
                flags, copies = E.HPC_FLAG_NO_PAGES, []
            else:
                for b, L in zip(dst, cut):
                    lens[b] = L
        else:
            hd.hpc_kv_compact(both.pool, both.table, both.copies)
            copies = op.compact(both.want)
        if check_each:
            both.check(flags, copies)
    both.check(flags)


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 9), (8, 10, 50), (40, 33, 600)])
@pytest.mark.parametrize("seed", range(3))
def test_sequences(shape, seed):
    play(Both(*shape), random.Random(seed), 40)


@pytest.mark.parametrize("shape", [(64, 65, 3000), (100, 300, 20000), (1000, 30, 30001)])
def test_sequences_of_several_ctas(shape):
    """More list entries than one CTA takes, and lists that are no multiple of anything."""
    play(Both(*shape), random.Random(7), 12)


def test_all_rows_and_no_rows():
    b = Both(5, 4, 30)
    lens = [256, 0, 1, 64, 65]
    hd.hpc_kv_extend(b.pool, b.table, None, ints(lens))
    op.extend(b.want, range(5), lens)
    b.check()
    none = ints([])
    hd.hpc_kv_extend(b.pool, b.table, none, none)
    hd.hpc_kv_free(b.pool, b.table, none)
    hd.hpc_kv_fork(b.pool, b.table, none, none, none, b.copies)
    b.check(copies=[])
    hd.hpc_kv_free(b.pool, b.table, None, ints([100, 0, 0, 64, 0]))
    op.free(b.want, range(5), [100, 0, 0, 64, 0])
    b.check()
    hd.hpc_kv_free(b.pool, b.table)
    op.free(b.want, range(5))
    b.check()


def test_a_shared_page_goes_back_with_its_last_holder():
    b = Both(6, 4, 12)
    hd.hpc_kv_extend(b.pool, b.table, ints([0]), ints([200]))
    op.extend(b.want, [0], [200])
    hd.hpc_kv_fork(b.pool, b.table, ints([0, 0, 0]), ints([5, 2, 1]), ints([200, 128, 65]), b.copies)
    b.check(copies=op.fork(b.want, [0, 0, 0], [5, 2, 1], [200, 128, 65]))
    for rows in ([0, 1], [5], [2]):  # the parent first, its pages live on
        hd.hpc_kv_free(b.pool, b.table, ints(rows))
        op.free(b.want, rows)
        b.check()
    assert b.pool.free_pages == 12


def test_rows_named_twice():
    b = Both(4, 6, 30)
    hd.hpc_kv_extend(b.pool, b.table, ints([1, 3, 1]), ints([200, 100, 300]))
    op.extend(b.want, [1, 3, 1], [200, 100, 300])
    b.check()
    hd.hpc_kv_free(b.pool, b.table, ints([1, 1, 3]), ints([64, 0, 100]))
    assert b.table.tolist() == [[-1] * 6, [-1] * 6, [-1] * 6, b.want["table"][3]]
    assert b.pool.state.tolist() == [28, 0, 0, 0]
    held = [p for p in b.want["table"][3] if p >= 0]
    assert sorted(b.pool.free_list[:28].tolist()) == sorted(set(range(30)) - set(held))
    # two children of one row: the first is born
    hd.hpc_kv_fork(b.pool, b.table, ints([3, 3]), ints([0, 0]), ints([70, 100]), b.copies)
    assert b.pool.flags == E.HPC_FLAG_BAD_SEQLEN and int(b.copies[0, 0]) == 1
    assert b.table[0].tolist()[0] == held[0] and int(b.pool.refs[held[0]]) == 2


def test_refused_rows_change_nothing():
    b = Both(4, 4, 9)
    lens = [130, 70, 0, 0]
    hd.hpc_kv_extend(b.pool, b.table, None, ints(lens))
    op.extend(b.want, range(4), lens)
    bad = E.HPC_FLAG_BAD_SEQLEN
    hd.hpc_kv_extend(b.pool, b.table, ints([4, -1, 2, 3]), ints([64, 64, 257, -5]))
    b.check(bad)
    hd.hpc_kv_free(b.pool, b.table, ints([99, 0, 1]), ints([0, -1, 300]))
    b.check(bad)
    # onto a row in use, from a row to itself, from a row that is born in the same call,
    # from outside, of more than there is (its third page is missing)
    for src, dst, n in (([0], [1], [64]), ([0], [0], [64]), ([0, 2], [2, 3], [64, 64]),
                        ([7], [2], [64]), ([0], [2], [10 ** 6])):
        hd.hpc_kv_fork(b.pool, b.table, ints(src), ints(dst), ints(n), b.copies)
        if len(src) == 2:
            op.fork(b.want, src[:1], dst[:1], n[:1])
            bad |= E.HPC_FLAG_BAD_PAGE
        b.check(bad)
    hd.hpc_kv_fork(b.pool, b.table, ints([1]), ints([3]), ints([129]), b.copies)
    b.check(bad, copies=[])


def test_pages_that_are_none_of_the_pools():
    b = Both(3, 4, 8)
    hd.hpc_kv_extend(b.pool, b.table, ints([0]), ints([100]))
    op.extend(b.want, [0], [100])
    b.table[1] = ints([3, 800, -7, 5])  # a page that none holds, one outside, no page
    hd.hpc_kv_free(b.pool, b.table, ints([1]))
    assert b.table[1].tolist() in ([-1, -1, -7, -1], [-1, -1, -1, -1])
    b.table[1] = -1
    b.check(E.HPC_FLAG_BAD_PAGE)
    b.table[1] = ints([800, 801, 802, 803])
    hd.hpc_kv_fork(b.pool, b.table, ints([1]), ints([2]), ints([200]), b.copies)
    assert b.table[2].tolist() == [-1] * 4
    b.table[1] = -1
    b.check(E.HPC_FLAG_BAD_PAGE, copies=[])


@pytest.mark.parametrize("in_place", [True, False])
def test_compaction_out_of_place_leaves_the_old_pool(in_place):
    b = Both(6, 8, 40)
    lens = [500, 20, 300, 64, 512, 1]
    hd.hpc_kv_extend(b.pool, b.table, None, ints(lens))
    op.extend(b.want, range(6), lens)
    hd.hpc_kv_free(b.pool, b.table, ints([0, 3]))
    op.free(b.want, [0, 3])
    if in_place:
        hd.hpc_kv_compact(b.pool, b.table, b.copies)
        b.check(copies=op.compact(b.want))
        return
    table, pool = torch.zeros_like(b.table), hd.PagePool(40)
    hd.hpc_kv_compact(b.pool, b.table, b.copies, table, pool)
    b.check()
    old, b.table, b.pool = b.pool, table, pool
    b.check(copies=op.compact(b.want))
    assert (old.marks == IDLE).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "block"])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_copies(kv, heads):
    gen = torch.Generator(device="cuda").manual_seed(heads)
    dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    width = 2 if kv == "bf16" else 1
    caches = [torch.randint(0, 256, (50, 64, heads, 128 * width), generator=gen, device="cuda",
                            dtype=torch.uint8) for _ in range(2)]
    scale = torch.rand((50, heads, 2, 4), generator=gen, device="cuda") if kv == "block" else None
    pairs = [(3, 40), (3, 41), (0, 49), (49 - 9, 1)]
    pairs[3] = (7, 1)
    copies = ints([[len(pairs), 0]] + [list(p) for p in pairs] + [[5, 6]] * 3)
    want = [c.clone() for c in caches] + [scale.clone() if scale is not None else None]
    for a, b in pairs:
        for t in want:
            if t is not None:
                t[b] = t[a]
    hd.hpc_kv_copy_pages(copies, *(c.view(dtype) for c in caches), scale)
    for got, t in zip(caches + [scale], want):
        assert t is None or torch.equal(got, t)
    # a count beyond the list's end, and pages outside the cache
    flags = ints([0])
    copies = ints([[1000, 0], [2, 50], [-1, 3], [4, 5]])
    for t in want:
        if t is not None:
            t[5] = t[4]
    hd.hpc_kv_copy_pages(copies, *(c.view(dtype) for c in caches), scale, flags)
    assert int(flags) == E.HPC_FLAG_BAD_PAGE
    for got, t in zip(caches + [scale], want):
        assert t is None or torch.equal(got, t)


def test_captured_on_a_stream_of_its_own():
    """Children that end, others that are forked and copied: captured once, replayed."""
    b = Both(12, 9, 60)
    lens = [500, 130] + [0] * 10
    hd.hpc_kv_extend(b.pool, b.table, None, ints(lens))
    op.extend(b.want, range(12), lens)
    k = torch.randn((60, 64, 2, 128), device="cuda").bfloat16()
    v = torch.randn((60, 64, 2, 128), device="cuda").bfloat16()
    src, dst, cut = ints([0, 1, 0]), ints([7, 3, 9]), ints([500, 100, 70])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        hd.hpc_kv_free(b.pool, b.table, dst)
        hd.hpc_kv_fork(b.pool, b.table, src, dst, cut, b.copies)
        hd.hpc_kv_copy_pages(b.copies, k, v)
    torch.cuda.synchronize()
    b.check()  # nothing has run
    want = op.fork(b.want, [0, 1, 0], [7, 3, 9], [500, 100, 70])
    for _ in range(3):
        graph.replay()
        b.check(copies=want)
        for a, c in want:
            assert torch.equal(k[a], k[c]) and torch.equal(v[a], v[c])
    # other lengths and parents, the same graph
    src.copy_(ints([1, 0, 0]))
    cut.copy_(ints([130, 0, 449]))
    op.free(b.want, [7, 3, 9])
    want = op.fork(b.want, [1, 0, 0], [7, 3, 9], [130, 0, 449])
    graph.replay()
    b.check(copies=want)


def test_lists_of_several_rounds():
    """More list entries than a cluster holds at once (131,072)."""
    play(Both(600, 501, 60000), random.Random(11), 8)


def test_a_rollback_into_a_shared_page_by_a_fork():
    """A child that goes back to a token inside a page that others hold: a fork of its
    first tokens gets a copy to write to, and the row itself then goes."""
    both = Both(3, 4, 20)
    hd.hpc_kv_extend(both.pool, both.table, ints([0]), ints([256]))
    op.extend(both.want, [0], [256])
    hd.hpc_kv_fork(both.pool, both.table, ints([0]), ints([1]), ints([256]), both.copies)
    both.check(copies=op.fork(both.want, [0], [1], [256]))
    hd.hpc_kv_fork(both.pool, both.table, ints([1]), ints([2]), ints([200]), both.copies)
    copies = op.fork(both.want, [1], [2], [200])
    both.check(copies=copies)
    assert copies == [(both.want["table"][0][3], both.want["table"][2][3])]
    hd.hpc_kv_free(both.pool, both.table, ints([1]))
    op.free(both.want, [1], [0])
    both.check()
    assert both.table[2, :3].tolist() == both.table[0, :3].tolist()
    assert both.table[2, 3] != both.table[0, 3]
