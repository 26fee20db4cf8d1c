"""What the windowed and block-scaled calls promise about maps, bins and repeats."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
import oracle
from _blocks import DTYPE, Case
from oracle import window as ow

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["e4m3", "block"])
@pytest.mark.parametrize("heads", [(8, 1), (8, 2), (32, 2)])
def test_more_bins_than_ctas_repeat_bit_for_bit(kv, heads):
    """Which CTA takes a bin is a race where there are more bins than CTAs; what
    each descriptor's partial holds is not.  Descriptors of several stages, an odd
    number of them per bin."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(4000, 20000, 32)]
    c = Case(kv, lens, *heads, 1, 15000, 5, seed=91).to_gpu()
    total = sum(-(-n // 64) for n in ow.planned_lengths(lens, c.bt.shape[1], 1, 15000, 5))
    bins = -(-total // 9)  # tiles per bin: 9
    ws = c.workspace(bins)
    first = None
    for _ in range(20):
        ws.part_o.zero_()
        ws.part_lse.zero_()
        out, _ = c.step(floor=1, fused=False, ws=ws)
        got = [t.view(torch.int32).clone() for t in (ws.part_o, ws.part_lse)]
        got.append(out.view(torch.int16).clone())
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b)
    assert int(hd.hpc_decode_read_meta(ws.tmap)[1]) == 9
    c.check(out)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "block"])
def test_a_map_of_another_window_is_refused(kv):
    """Every window, sinks and q_len but the map's own, also where they are far
    apart (200 and 4 against 15885 and 2599)."""
    c = Case(kv, [900, 64, 300], 8, 2, 1, 200, 4, seed=92, poison=False).to_gpu()
    ws = c.workspace()
    hd.hpc_decode_plan_win(c.sl, 2, c.bt.shape[1], ws.num_ctas, 2, ws.tmap, kv_dtype=DTYPE[kv],
                           window=200, sinks=4)
    out = torch.zeros((3, 1, 8, 128), dtype=torch.bfloat16, device="cuda")

    def attn(window, sinks):
        hd.hpc_decode_attn_win(c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, c.bt, c.sl, 8, 2, 1,
                               window, sinks, c.sm, ws.tmap, ws.part_o, ws.part_lse, out,
                               ws.unit_done)

    attn(200, 4)
    c.check(out)
    for window, sinks in ((15885, 2599), (20874, 17266), (201, 4), (200, 5), (4, 200), (0, 0)):
        with pytest.raises(hd.HpcError):
            attn(window, sinks)
    torch.cuda.synchronize()
    # and a map of one query per request for two
    c2 = Case(kv, [900, 64, 300], 8, 2, 2, 200, 4, seed=92, poison=False).to_gpu()
    ws2 = c2.workspace()
    hd.hpc_decode_plan_win(c.sl, 2, c.bt.shape[1], ws.num_ctas, 2, ws2.tmap, kv_dtype=DTYPE[kv],
                           q_len=1, window=200, sinks=4)
    out2 = torch.zeros((3, 2, 8, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hd.HpcError):
        hd.hpc_decode_attn_win(c2.q, c2.qs, c2.k, c2.v, c2.ks, c2.vs, c2.scale, c2.bt, c2.sl, 8, 2,
                               2, 200, 4, c2.sm, ws2.tmap, ws2.part_o, ws2.part_lse, out2,
                               ws2.unit_done)


@pytest.mark.parametrize("kv", ["e4m3", "block"])
def test_a_map_of_head_pairs_on_the_host(kv):
    """to_host of a map whose units are pairs of heads: the pairs' counts, and nothing
    that an earlier plan left behind them."""
    lens = [700, 64, 0, 1200, 300]
    c = Case(kv, lens, 8, 4, 1, 500, 4, seed=93, poison=False).to_gpu()
    ws = c.workspace(40)
    hd.hpc_decode_plan(c.sl, 4, c.bt.shape[1], 40, 1, ws.tmap)  # single heads
    hd.hpc_decode_plan_win(c.sl, 4, c.bt.shape[1], 40, 1, ws.tmap, kv_dtype=DTYPE[kv],
                           window=500, sinks=4)
    torch.cuda.synchronize()
    got = ws.tmap.to_host()
    ref = oracle.assign_closed_form(ow.planned_lengths(lens, c.bt.shape[1], 1, 500, 4), 2, 40, 1)
    for name in ("total_tiles", "budget", "num_desc", "desc", "bin_ptr", "chunk_count",
                 "chunk_off"):
        assert got[name] == getattr(ref, name), name
