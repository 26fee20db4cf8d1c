"""Maps that a call refuses (no GPU: fake, never-dereferenced device pointers)."""

import ctypes

import pytest

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as E
from test_abi_window_cpu import FAKE, attn, fake_map


@pytest.fixture(scope="module", autouse=True)
def built():
    from load_balanced_paged_assign_gb300 import _build
    _build.build()


def window_map(q_len=1, window=200, sinks=4, **kw):
    m = fake_map(**kw)
    m.q_len, m.window, m.sinks = q_len, window, sinks
    return m


def test_a_window_is_checked_exactly():
    for q_len, window, sinks in ((1, 15885, 2599), (1, 20874, 17266), (1, 201, 4), (1, 200, 5),
                                 (1, 4, 200), (2, 200, 4), (1, 0, 0)):
        assert attn(q_len=q_len, window=window, sinks=sinks, m=window_map()) == E.HPC_ERR_ARG
    # head pairs or not goes by the cache's type and heads: two KV heads of E4M3 are one
    kw = dict(Hq=8, Hkv=2, dtype=1, qs=FAKE, window=200, sinks=4)
    assert attn(m=window_map(Hkv=2, persistent=1), **kw) == E.HPC_ERR_ARG
    assert attn(m=window_map(Hkv=2, persistent=3), **dict(kw, dtype=0, qs=None)) == E.HPC_ERR_ARG


def test_the_combine_takes_the_maps_query_count():
    m = window_map(q_len=2)
    assert hd.lib().hpc_decode_combine_mq(FAKE, FAKE, ctypes.byref(m), 4, 8, 1, 128, 1, FAKE,
                                          None) == E.HPC_ERR_ARG
    m = window_map(q_len=1)
    assert hd.lib().hpc_decode_combine_mq(FAKE, FAKE, ctypes.byref(m), 4, 8, 1, 128, 2, FAKE,
                                          None) == E.HPC_ERR_ARG


def test_to_host_of_a_map_of_head_pairs():
    """Units are pairs of heads: half as many counts, none left from an earlier plan."""
    m = E.TaskMap(3, 4, 20, 9, device="cpu")
    m.chunk_count[:] = 7
    m.c.B, m.c.Hkv, m.c.num_ctas, m.c.persistent = 3, 4, 8, 1
    assert len(m.to_host()["chunk_count"]) == len(m.to_host()["chunk_off"]) == 12
    m.c.persistent = 3
    assert len(m.to_host()["chunk_count"]) == len(m.to_host()["chunk_off"]) == 6


@pytest.mark.parametrize("kv", [E.HPC_KV_BF16, E.HPC_KV_FP8_E4M3, E.HPC_KV_E4M3_BLOCK])
@pytest.mark.parametrize("heads", [1, 2, 3, 4])
def test_a_workspace_has_room_for_the_descriptors_its_calls_make(kv, heads):
    """num_ctas + B Hkv of them; head pairs (8-bit caches, an even number of heads)
    take the room of two: 2 num_ctas + B Hkv, and nothing else does."""
    ws = hd.Workspace(5, 8 * heads, heads, num_ctas=30, kv_dtype=kv, device="cpu")
    pairs = kv != E.HPC_KV_BF16 and heads % 2 == 0
    assert ws.tmap.cap_desc == 30 * (2 if pairs else 1) + 5 * heads
    assert ws.part_o.shape == (ws.tmap.cap_desc, 8, 128)


def test_scales_that_are_infinite_once_multiplied():
    """sm_scale * log2(e) (* k_scale) past fp32's range: scores of zero would be NaN."""
    m = dict(m=window_map())
    assert attn(window=200, sinks=4, sm=3e38, **m) == E.HPC_ERR_ARG
    assert attn(dtype=2, kvs=FAKE, qs=FAKE, sm=3e38) == E.HPC_ERR_ARG

    def prompt(sm):
        return hd.lib().hpc_prefill_attn_win(FAKE, FAKE, FAKE, 100, FAKE, 8, FAKE, 0, 8, 2, 128,
                                             300, 128, 4, sm, FAKE, None, None)

    assert prompt(3e38) == E.HPC_ERR_ARG and prompt(2e38) == E.HPC_OK
