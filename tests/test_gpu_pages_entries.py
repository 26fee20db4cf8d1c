"""Compaction over a table with entries that name no page of the pool's."""

import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as E
from oracle import pages as op
from test_gpu_pages import IDLE, Both, ints

pytestmark = pytest.mark.gpu


def fragmented(B, cols, pages):
    """A pool with holes: rows of all lengths, every third one gone."""
    b = Both(B, cols, pages)
    lens = [1 + (97 * r) % (64 * cols) for r in range(B)]
    hd.hpc_kv_extend(b.pool, b.table, None, ints(lens))
    assert op.extend(b.want, range(B), lens)
    gone = list(range(0, B, 3))
    hd.hpc_kv_free(b.pool, b.table, ints(gone))
    op.free(b.want, gone)
    b.check()
    return b


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("shape", [(6, 8, 40), (100, 70, 5000)])
def test_compaction_flags_entries_that_name_no_held_page(in_place, shape):
    """Outside the pool, or a page that no entry holds (in front of the last held one and
    behind it): the entry becomes -1, or two rows would name one page later.  The rest is as
    without them, and the marks are left idle."""
    b = fragmented(*shape)
    pages = shape[2]
    live = sum(r > 0 for r in b.want["refs"])
    near = next(p for p in range(live) if b.want["refs"][p] == 0)
    far = next(p for p in range(pages - 1, live - 1, -1) if b.want["refs"][p] == 0)
    row = ints([near, far, pages, 2 ** 31 - 1, -7])  # row 0 is empty; -7: no page
    b.table[0, :5] = row
    table, pool = (b.table, b.pool) if in_place else (torch.zeros_like(b.table), hd.PagePool(pages))
    hd.hpc_kv_compact(b.pool, b.table, b.copies, table, pool)
    copies = op.compact(b.want)
    assert table[0, :5].tolist() in ([-1, -1, -1, -1, -7], [-1] * 5)
    if not in_place:  # the old table and pool are as they were
        assert torch.equal(b.table[0, :5], row)
        assert b.pool.flags == 0 and (b.pool.marks == IDLE).all()
    table[0, :5] = -1
    b.table, b.pool = table, pool
    b.check(E.HPC_FLAG_BAD_PAGE, copies=copies)


def test_flags_of_the_old_pool_go_with_it():
    b = fragmented(6, 8, 40)
    b.pool.state[1] = E.HPC_FLAG_NO_PAGES
    table, pool = torch.zeros_like(b.table), hd.PagePool(40)
    hd.hpc_kv_compact(b.pool, b.table, b.copies, table, pool)
    copies = op.compact(b.want)
    b.table, b.pool = table, pool
    b.check(E.HPC_FLAG_NO_PAGES, copies=copies)
    b.table[0, 0] = 39
    hd.hpc_kv_compact(b.pool, b.table, b.copies)
    b.check(E.HPC_FLAG_NO_PAGES | E.HPC_FLAG_BAD_PAGE, copies=[])
