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


def test_write_read_and_decode_captured_on_another_stream():
    """The cache written, read back and attended over, captured together on a stream of
    its own and replayed with other rows: what the calls one by one leave."""
    from _blocks import E4M3, Prologue
    tokens = [(r, p) for r, n in enumerate((70, 16, 33)) for p in range(n)]
    pro = Prologue(tokens, 8, 2, B=3, max_pages=2, seed=94)
    other = Prologue(tokens, 8, 2, B=3, max_pages=2, seed=95)
    lens = torch.tensor([70, 16, 33], dtype=torch.int32, device="cuda")
    table = torch.from_numpy(pro.table).cuda()
    ws = hd.Workspace(3, 8, 2, kv_dtype=hd.HPC_KV_E4M3_BLOCK)
    last = torch.tensor([69, 85, 118], device="cuda")  # the requests' last tokens
    pos, req = torch.from_numpy(pro.pos).cuda(), torch.from_numpy(pro.req).cuda()
    wq, wk = pro.wq.cuda(), pro.wk.cuda()

    def buffers():
        k, v = (torch.from_numpy(c.copy()).cuda().view(E4M3) for c in pro.codes0)
        b = dict(qkv=pro.full.cuda(), k=k, v=v, s=torch.from_numpy(pro.scale0.copy()).cuda(),
                 q=torch.zeros((pro.N, 8, 128), device="cuda").to(E4M3),
                 qs=torch.zeros((pro.N, 8), device="cuda"),
                 out=torch.zeros((3, 1, 8, 128), dtype=torch.bfloat16, device="cuda"))
        b["ko"] = torch.zeros((pro.P, 64, 2, 128), dtype=torch.bfloat16, device="cuda")
        b["vo"] = torch.zeros_like(b["ko"])
        b["q1"], b["qs1"] = b["q"][:3].clone(), b["qs"][:3].clone()
        return b

    def run(b, stream=None):
        hd.hpc_rope_norm_block(b["qkv"], wq, wk, pos, req, 8, 2, table, b["k"], b["v"], b["s"],
                               b["q"], b["qs"], stream=stream)
        hd.hpc_kv_read_block(b["k"], b["v"], b["s"], table, None, lens, 2, b["ko"], b["vo"], table,
                             stream=stream)
        b["q1"].view(torch.uint8).copy_(b["q"].view(torch.uint8)[last])
        b["qs1"].copy_(b["qs"][last])
        hd.hpc_decode_step_win(b["q1"], b["qs1"], b["k"], b["v"], 1.0, 1.0, b["s"], table, lens, 8,
                               2, 1, 40, 4, 128 ** -0.5, ws.num_ctas, 2, ws.tmap, ws.part_o,
                               ws.part_lse, b["out"], unit_done=ws.unit_done, stream=stream)

    def same(a, b):
        torch.cuda.synchronize()
        for name in a:
            assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name

    eager, replayed, named = buffers(), buffers(), buffers()
    run(eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(named, stream=side)
    same(eager, named)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(replayed)
    graph.replay()
    same(eager, replayed)
    for b in (eager, replayed):
        b["qkv"].copy_(other.full)
    run(eager)
    graph.replay()
    same(eager, replayed)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "block"])
def test_no_requests(kv):
    """An empty batch: nothing is written, and the workspace serves the next step."""
    c = Case(kv, [200, 64], 8, 2, 1, 100, 4, seed=96, poison=False).to_gpu()
    ws = c.workspace()
    out = torch.full((2, 1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    none = [None if t is None else t[:0] for t in (c.q, c.qs, c.bt, c.sl)]
    for done in (ws.unit_done, None):
        hd.hpc_decode_step_win(none[0], none[1], c.k, c.v, c.ks, c.vs, c.scale, none[2], none[3],
                               8, 2, 1, 100, 4, c.sm, ws.num_ctas, 2, ws.tmap, ws.part_o,
                               ws.part_lse, out, unit_done=done)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and ws.tmap.to_host()["num_desc"] == 0
    got, _ = c.step(ws=ws)
    c.check(got)
    if kv == "bf16":
        hd.hpc_prefill_attn_win(none[0], c.k, c.v, none[2], none[3], 8, 2, 1, 100, 4, c.sm, out)
        torch.cuda.synchronize()
        assert (out == 7.0).all()
