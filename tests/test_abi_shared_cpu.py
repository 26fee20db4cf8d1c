"""Host-side refusals of the shared-prefix entry points (no GPU: fake,
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


def capacity(B=4, Hq=8, Hkv=1, q_len=1, groups=2, ctas=152, sizes=True):
    out = (ctypes.c_int64 * 3)()
    st = hd.lib().hpc_decode_shared_capacity(B, Hq, Hkv, q_len, groups, ctas,
                                             out if sizes else None)
    return st if st else list(out)


def test_capacities():
    assert capacity(Hq=17) == UNS and capacity(Hq=6, Hkv=4) == UNS and capacity(q_len=3) == UNS
    assert capacity(B=-1) == ARG and capacity(Hq=0) == ARG and capacity(Hkv=0) == ARG
    assert capacity(q_len=0) == ARG and capacity(groups=-1) == ARG and capacity(sizes=False) == ARG
    assert capacity(ctas=1) == ARG and capacity(ctas=(1 << 16) + 1) == UNS
    assert capacity(B=8193) == UNS and capacity(groups=4097) == UNS
    cap, ints, slots = capacity()
    assert cap == 2 * 152 + 4 and slots == 2 * (2 + 152)
    # no two requests, no heads
    assert capacity(B=1)[2] == 1 and capacity(groups=0)[2] == 1
    # 64 requests of 3 rows in tiles of 42 tokens: at most 32 groups of a pair of tiles, and
    # a pair more for each 84 tokens
    assert capacity(B=64, Hq=3, groups=100)[2] == 2 * (32 + 64 // 84 + 152)


def shared_map(**kw):
    tail = E.hpc_task_map(FAKE, FAKE, FAKE, FAKE, FAKE, 1000, 200, 64)
    f = dict(head=FAKE, head_o=FAKE, head_lse=FAKE, cap_head=10 ** 6, cap_slots=10 ** 5)
    for k, v in kw.items():
        if k in f or k in ("Hq", "num_groups", "kv_dtype"):
            f[k] = v
        else:
            setattr(tail, k, v)
    return E.hpc_shared_map(tail, **f)


def plan(m=None, B=4, Hq=8, Hkv=1, max_pages=32, starts=FAKE, pages=FAKE, groups=2, ctas=132,
         floor=2, dtype=0, q_len=1, lens=FAKE):
    m = m or shared_map()
    return hd.lib().hpc_decode_plan_shared(lens, B, Hq, Hkv, max_pages, starts, pages, groups, ctas,
                                           floor, dtype, q_len, ctypes.byref(m), None)


def test_plan_refusals():
    assert plan(lens=None) == ARG and plan(starts=None) == ARG and plan(pages=None) == ARG
    assert plan(max_pages=0) == ARG and plan(floor=-1) == ARG and plan(floor=1 << 27) == ARG
    assert plan(dtype=3) == ARG and plan(ctas=1) == ARG
    assert plan(max_pages=1 << 24) == UNS and plan(max_pages=1 << 20, B=4096) == UNS
    assert plan(q_len=2, Hq=9) == UNS
    for name in ("desc", "bin_ptr", "chunk_count", "chunk_off", "meta", "head", "head_o",
                 "head_lse"):
        assert plan(shared_map(**{name: None})) == ARG
    assert plan(shared_map(head=FAKE + 4)) == ARG and plan(shared_map(head_o=FAKE + 16)) == ARG
    assert plan(shared_map(cap_desc=267)) == ROOM and plan(shared_map(cap_bins=132)) == ROOM
    assert plan(shared_map(cap_units=3)) == ROOM and plan(shared_map(cap_slots=100)) == ROOM
    assert plan(shared_map(cap_head=100)) == ROOM
    assert hd.lib().hpc_decode_plan_shared(FAKE, 4, 8, 1, 32, FAKE, FAKE, 2, 132, 2, 0, 1, None,
                                           None) == ARG


def planned(dtype=0, heads=1, **kw):
    f = dict(B=4, Hkv=1, num_ctas=132, persistent=5 | (heads - 1) << 1, max_pages=32, q_len=1,
             Hq=8, num_groups=2, kv_dtype=dtype) | kw
    return shared_map(**f)


def attn(m=None, q=FAKE, qs=None, k=FAKE, v=FAKE, pages=10, ks=1.0, vs=1.0, kvs=None, dtype=0,
         bt=FAKE, max_pages=32, lens=FAKE, B=4, Hq=8, Hkv=1, D=128, q_len=1, sm=0.088, po=FAKE,
         pl=FAKE, out=FAKE):
    m = m or planned(dtype)
    return hd.lib().hpc_decode_attn_shared(q, qs, k, v, pages, ks, vs, kvs, dtype, bt, max_pages,
                                           lens, B, Hq, Hkv, D, q_len, sm, ctypes.byref(m), po, pl,
                                           out, None)


def test_attention_refusals():
    assert attn(D=64) == UNS and attn(pages=0) == ARG
    for name in ("q", "k", "v", "bt", "lens", "po", "pl", "out"):
        assert attn(**{name: None}) == ARG, name
    for name in ("q", "k", "v", "po", "out"):
        assert attn(**{name: FAKE + 8}) == ARG, name
    assert attn(kvs=FAKE) == ARG and attn(dtype=2, qs=FAKE) == ARG
    assert attn(dtype=2, qs=FAKE, kvs=FAKE + 4) == ARG and attn(dtype=1) == ARG
    assert attn(sm=float("nan")) == ARG and attn(sm=3e38) == ARG
    assert attn(dtype=1, qs=FAKE, ks=float("inf")) == ARG
    assert attn(dtype=1, qs=FAKE, vs=float("nan")) == ARG
    # maps of another batch, another kind, or no plan of this call's
    for kw in (dict(B=5), dict(Hkv=2, Hq=16), dict(q_len=2), dict(max_pages=33), dict(Hq=4),
               dict(kv_dtype=1), dict(persistent=1), dict(persistent=7), dict(persistent=0)):
        assert attn(planned(**kw)) == ARG, kw
    # 8-bit caches of an even number of heads: descriptors of pairs
    assert attn(planned(1, Hkv=2, Hq=16), qs=FAKE, dtype=1, Hkv=2, Hq=16) == ARG


def test_other_calls_refuse_the_tails_map():
    m = planned().tail
    assert hd.lib().hpc_decode_attn(FAKE, None, FAKE, FAKE, 10, 1.0, 1.0, 0, FAKE, 32, FAKE, 4, 8,
                                    1, 128, 0.088, ctypes.byref(m), FAKE, FAKE, None) == ARG
    assert hd.lib().hpc_decode_combine(FAKE, FAKE, ctypes.byref(m), 4, 8, 1, 128, FAKE,
                                       None) == ARG
    assert hd.lib().hpc_decode_attn_win(FAKE, FAKE, FAKE, FAKE, 10, 1.0, 1.0, FAKE, 2, FAKE, 32,
                                        FAKE, 4, 8, 1, 128, 1, 0, 0, 0.088, ctypes.byref(m), FAKE,
                                        FAKE, FAKE, FAKE, None) == ARG


def test_refusals_of_the_binding():
    i32 = dict(dtype=torch.int32)
    ws = hd.SharedWorkspace(2, 8, 1, 1, num_ctas=4, device="cpu")
    q = torch.zeros((2, 1, 8, 128), dtype=torch.bfloat16)
    k = torch.zeros((6, 64, 1, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 3), **i32), torch.ones(2, **i32)
    starts, pages, out = torch.tensor([0, 2], **i32), torch.ones(1, **i32), torch.zeros_like(q)

    def step(q=q, k=k, table=table, lens=lens, starts=starts, pages=pages, ws=ws, out=out, q_len=1):
        hd.hpc_decode_step_shared(q, None, k, k, 1.0, 1.0, None, table, lens, starts, pages, 8, 1,
                                  q_len, 0.088, 2, ws, out)

    for kw, match in ((dict(q=q.float()), "q is"), (dict(k=k[:, :, :, :64]), "k_cache"),
                      (dict(table=table[:1]), "block_table"), (dict(starts=starts.long()), "starts"),
                      (dict(starts=starts[:1]), "one more"), (dict(pages=pages[:0]), "one more"),
                      (dict(out=out[:1]), "q or out"), (dict(q_len=2), "q or out"),
                      (dict(starts=torch.zeros(3, **i32), pages=torch.zeros(2, **i32)), "room")):
        with pytest.raises(ValueError, match=match):
            step(**kw)
    with pytest.raises(ValueError, match="no SharedWorkspace"):
        hd.hpc_decode_plan_shared(lens, starts, pages, 8, 1, 1, 3, 2, hd.Workspace)
    with pytest.raises(hd.HpcError):  # more requests than the workspace holds
        hd.hpc_decode_plan_shared(torch.ones(64, **i32), starts, pages, 8, 1, 1, 3, 2, ws)


def test_shapes_whose_costs_leave_32_bits():
    """32 a unit: 16,384 KV heads times 4096 pairs of requests and more; and KV heads that the
    plan's quotients do not hold."""
    assert capacity(B=8192, Hq=16384, Hkv=16384, groups=4096) == UNS
    assert type(capacity(B=8192, Hq=4096, Hkv=4096, groups=4096)) is list
    assert type(capacity(B=8192, Hq=16384, Hkv=16384, groups=0)) is list
    assert capacity(B=1, Hq=1 << 20, Hkv=1 << 20) == UNS
    assert type(capacity(B=1, Hq=(1 << 20) - 1, Hkv=(1 << 20) - 1)) is list
    assert plan(shared_map(cap_desc=1 << 40, cap_head=1 << 40, cap_slots=1 << 40,
                           cap_units=1 << 30), B=8192, Hq=16384, Hkv=16384, max_pages=1,
                groups=4096) == UNS
