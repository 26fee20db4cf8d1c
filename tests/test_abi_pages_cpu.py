"""Host-side refusals of the page pool's entry points (no GPU: fake,
never-dereferenced device pointers, and CPU tensors for the binding)."""

import ctypes

import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as E

FAKE = 0x10000
ARG, UNS, ROOM = E.HPC_ERR_ARG, E.HPC_ERR_UNSUPPORTED, E.HPC_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built():
    from load_balanced_paged_assign_gb300 import _build
    _build.build()


def pool(**kw):
    f = dict(refs=FAKE, free_list=FAKE, state=FAKE, marks=FAKE, num_pages=100) | kw
    return ctypes.byref(E.hpc_page_pool(**f))


@pytest.mark.parametrize("fn", ["hpc_kv_free", "hpc_kv_extend"])
def test_refusals_of_rows(fn):
    def call(p=None, table=FAKE, B=4, cols=8, rows=FAKE, lens=FAKE, n=3):
        return getattr(hd.lib(), fn)(p or pool(), table, B, cols, rows, lens, n, None)

    assert call(n=0) == E.HPC_OK and call(n=0, table=None) == E.HPC_OK
    for name in ("refs", "free_list", "state", "marks"):
        assert call(pool(**{name: None})) == ARG
    assert call(pool(num_pages=0)) == ARG
    assert call(pool(num_pages=1 << 30)) == UNS
    assert call(table=None) == ARG
    assert call(B=-1) == ARG and call(n=-1) == ARG and call(cols=0) == ARG
    assert call(B=HPC_MAX + 1) == UNS and call(n=HPC_MAX + 1) == UNS
    assert call(cols=1 << 24) == UNS  # token indices
    assert call(n=16384, B=16384, cols=1 << 16) == UNS  # list entries
    assert call(rows=None, n=5) == ARG  # all rows, but there are four
    if fn == "hpc_kv_extend":
        assert call(lens=None) == ARG


HPC_MAX = 16384


def test_refusals_of_forks_and_compactions():
    def fork(p=None, src=FAKE, dst=FAKE, lens=FAKE, n=3, copies=FAKE, cap=3, B=4):
        return hd.lib().hpc_kv_fork(p or pool(), FAKE, B, 8, src, dst, lens, n, copies, cap, None)

    assert fork(cap=2) == ROOM and fork(cap=-1) == ARG and fork(copies=None) == ARG
    assert fork(src=None) == ARG and fork(dst=None) == ARG and fork(lens=None) == ARG
    assert fork(B=HPC_MAX + 1) == UNS

    def compact(p=None, table=FAKE, B=4, cols=8, copies=FAKE, cap=50, to=FAKE, q=None):
        return hd.lib().hpc_kv_compact(p or pool(), table, B, cols, copies, cap, to, q or pool(),
                                       None)

    assert compact(cap=49) == ROOM and compact(cap=-1) == ARG and compact(copies=None) == ARG
    assert compact(table=None) == ARG and compact(to=None) == ARG
    assert compact(q=pool(num_pages=99)) == ARG
    assert compact(q=pool(refs=FAKE * 2)) == ARG  # two pools that share their stack
    assert compact(q=pool(refs=FAKE * 2, free_list=FAKE * 2)) == ARG
    assert compact(q=pool(state=None)) == ARG
    assert compact(B=-1) == ARG and compact(cols=0) == ARG


def test_refusals_of_copies():
    def call(copies=FAKE, cap=5, k=FAKE, v=FAKE, sc=None, dtype=0, pages=10, Hkv=2, D=128):
        return hd.lib().hpc_kv_copy_pages(copies, cap, k, v, sc, dtype, pages, Hkv, D, None, None)

    assert call(cap=0) == E.HPC_OK
    assert call(copies=None) == ARG and call(k=None) == ARG and call(v=None) == ARG
    assert call(k=FAKE + 8) == ARG and call(v=FAKE + 8) == ARG
    assert call(sc=FAKE) == ARG  # scales of a cache that has none
    assert call(dtype=2) == ARG and call(dtype=2, sc=FAKE + 8) == ARG and call(dtype=3) == ARG
    assert call(D=64) == UNS and call(Hkv=1 << 20) == UNS
    assert call(pages=0) == ARG and call(Hkv=0) == ARG and call(cap=-1) == ARG


def test_refusals_of_the_binding():
    i32 = dict(dtype=torch.int32)
    p = hd.PagePool(10, device="cpu")
    table, rows = torch.full((4, 3), -1, **i32), torch.zeros(2, **i32)
    copies = torch.zeros((6, 2), **i32)
    with pytest.raises(ValueError, match="int32 arrays"):
        hd.PagePool.of(p.refs, p.free_list[:9], p.state)
    with pytest.raises(ValueError, match="int32 arrays"):
        hd.PagePool.of(p.refs.long(), p.free_list, p.state)
    with pytest.raises(ValueError, match="no PagePool"):
        hd.hpc_kv_free(None, table)
    with pytest.raises(ValueError, match="matrix"):
        hd.hpc_kv_free(p, table[0])
    with pytest.raises(ValueError, match="not contiguous"):
        hd.hpc_kv_free(p, table.t())
    with pytest.raises(ValueError, match="rows is torch.int64"):
        hd.hpc_kv_free(p, table, rows.long())
    with pytest.raises(ValueError, match="keep has not 2"):
        hd.hpc_kv_free(p, table, rows, torch.zeros(3, **i32))
    with pytest.raises(ValueError, match="lens has not 2"):
        hd.hpc_kv_extend(p, table, rows, None)
    with pytest.raises(ValueError, match="are needed"):
        hd.hpc_kv_fork(p, table, rows, rows, None, copies)
    with pytest.raises(ValueError, match="dst has not 2"):
        hd.hpc_kv_fork(p, table, rows, rows[:1], rows, copies)
    with pytest.raises(ValueError, match="capacity"):
        hd.hpc_kv_fork(p, table, rows, rows, rows, copies.view(-1))
    with pytest.raises(ValueError, match="out_table"):
        hd.hpc_kv_compact(p, table, copies, table[:3].contiguous())
    k = torch.zeros((10, 64, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="v_cache"):
        hd.hpc_kv_copy_pages(copies, k, k[:9])
    with pytest.raises(ValueError, match="kv_scale"):
        hd.hpc_kv_copy_pages(copies, k, k, torch.zeros((10, 2, 2, 5)))
    with pytest.raises(ValueError, match="E4M3"):
        hd.hpc_kv_copy_pages(copies, k, k, torch.zeros((10, 2, 2, 4)))
