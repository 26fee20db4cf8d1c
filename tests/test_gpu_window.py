"""Windowed attention with sinks (decode and prefill) on every cache type, and
decode over the block-scaled cache, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
import oracle
from _blocks import DTYPE, Case, check_attention
from _gpu import device_ctas
from load_balanced_paged_assign_gb300.workloads import Workload, make_batch
from oracle import window as ow

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "block"]
# (Hq, Hkv, q_len): query rows per KV head on both sides of 8
HEADS = [(8, 1, 1), (2, 2, 1), (16, 1, 1), (6, 2, 2), (8, 1, 2), (3, 1, 5), (32, 2, 1), (16, 4, 3),
         (10, 2, 3), (9, 3, 4), (12, 6, 8)]
# (window, sinks): inside a tile, tile edges, sinks of several tiles, windows
# beyond every length, a window of one, sinks beyond the lengths
WINDOWS = [(1, 0), (5, 3), (64, 0), (65, 64), (100, 65), (130, 200), (700, 1), (10000, 4),
           (33, 5000)]
LENS = [1, 0, 63, 64, 65, 129, 190, 500, 777, 1000, 2, 2300]


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("win", WINDOWS)
@pytest.mark.parametrize("heads", [0, 3, 4, 7])
def test_windowed_decode(kv, win, heads):
    hq, hkv, n = HEADS[heads]
    c = Case(kv, LENS, hq, hkv, n, *win, seed=100 + heads).to_gpu()
    for ctas, fused in ((13, True), (0, True), (0, False)):
        got, _ = c.step(ctas=ctas, fused=fused)
        c.check(got)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("heads", range(len(HEADS)))
def test_head_layouts(kv, heads):
    hq, hkv, n = HEADS[heads]
    c = Case(kv, LENS, hq, hkv, n, 96, 17, seed=200 + heads).to_gpu()
    got, _ = c.step()
    c.check(got)


@pytest.mark.parametrize("heads", range(len(HEADS)))
@pytest.mark.parametrize("spread", [0.0, 4.0, 40.0])
def test_block_scaled_decode(heads, spread):
    """The whole context; block sizes from equal to 2^40 apart."""
    hq, hkv, n = HEADS[heads]
    c = Case("block", LENS + [4000], hq, hkv, n, 0, 0, seed=300 + heads, spread=spread).to_gpu()
    for ctas, fused in ((11, True), (0, True), (0, False)):
        got, _ = c.step(ctas=ctas, fused=fused)
        c.check(got)


def test_block_scales_of_any_size():
    """Scales that are no powers of two, zero, tiny and huge: the weights stay in
    range, and a zero V scale contributes nothing."""
    c = Case("block", [300, 64, 1000], 8, 1, 1, 0, 0, seed=41, poison=False)
    rng = np.random.default_rng(5)
    s = c.scale.numpy()
    s[:, :, 0] *= rng.uniform(0.5, 1.0, s[:, :, 0].shape)
    s[:, :, 1] = np.exp2(rng.uniform(-100, 100, s[:, :, 1].shape))
    s[:, :, 1][rng.random(s[:, :, 1].shape) < 0.2] = 0.0
    from oracle import block_cache as bc
    c.kf, c.vf = (bc.values(x.view(torch.uint8).numpy(), s, i) for i, x in enumerate((c.k, c.v)))
    # the largest outputs fit BF16 and fp32: 2^100 * 448
    got, _ = c.to_gpu().step()
    c.check(got)
    c.scale[:, :, 1] = 0.0
    got, _ = c.step()
    assert not got.float().abs().sum()


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -126, 2.0 ** -100])
def test_tiny_v_scales_over_many_tokens(scale):
    """In units of a V scale of 2^-100 the softmax's sum over 24,000 tokens whose
    weights stand 2^11.2 above the first ones' (the reference stays where those
    put it) would pass 2^128: 2^(100 + 3 + 11.2) * 12,000 for each half."""
    c = Case("block", [24000], 8, 1, 1, 0, 0, seed=42, poison=False)
    rows = c.table[0]
    c.k.view(torch.uint8).zero_()
    c.k.view(torch.uint8)[torch.from_numpy(rows[4:]), :, :, 0] = 0x38  # 1.0 from token 256 on
    c.q.view(torch.uint8).zero_()
    c.q.view(torch.uint8)[..., 0] = 0x38
    c.qs.fill_(11.2 * np.log(2.0) / c.sm)
    s = c.scale.numpy()
    s[:, :, 0] = 1.0
    s[:, :, 1] = scale
    c.qf = c.q.float().double().numpy() * c.qs.double().numpy()[..., None]
    from oracle import block_cache as bc
    c.kf, c.vf = (bc.values(x.view(torch.uint8).numpy(), s, i) for i, x in enumerate((c.k, c.v)))
    got, _ = c.to_gpu().step(ctas=1)
    if scale < 2.0 ** -100:  # counts as zero
        assert not got.float().abs().sum()
        return
    ref, mass = c.reference()
    # scaled up by 2^90 (exactly), where the bound's absolute parts mean nothing
    up = 2.0 ** 90
    check_attention(got.double() * up, ref * up, mass * up, "block")


def test_static_map_of_an_odd_number_of_heads():
    """Without a window and without head pairs a map of equal splits serves too."""
    c = Case("block", [300, 1, 0, 700], 6, 3, 1, 0, 0, seed=43).to_gpu()
    ws = hd.Workspace(4, 6, 3, num_splits=5, kv_dtype=DTYPE["block"])
    hd.hpc_decode_plan_static(c.sl, 3, c.bt.shape[1], 5, ws.tmap)
    out = torch.full((4, 1, 6, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    args = (c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, c.bt, c.sl, 6, 3, 1, 0, 0, c.sm, ws.tmap,
            ws.part_o, ws.part_lse)
    hd.hpc_decode_attn_win(*args, out, ws.unit_done)
    c.check(out)
    two = torch.full_like(out, float("nan"))
    hd.hpc_decode_attn_win(*args)
    hd.hpc_decode_combine_mq(ws.part_o, ws.part_lse, ws.tmap, 4, 6, 3, 1, two)
    c.check(two)
    assert not int(torch.count_nonzero(ws.unit_done))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2])
def test_without_a_window_it_is_the_plain_step(kv, n):
    c = Case(kv, [1, 64, 700, 3000, 0], 8, 1, n, 0, 0, seed=7, poison=False).to_gpu()
    got, ws = c.step()
    out = torch.full_like(got, float("nan"))
    hd.hpc_decode_step_mq(c.q, c.qs, c.k, c.v, c.ks, c.vs, c.bt, c.sl, 8, 1, n, c.sm, ws.num_ctas,
                          2, 0, ws.tmap, ws.part_o, ws.part_lse, out, unit_done=ws.unit_done)
    assert torch.equal(got.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_window_beyond_every_length_is_the_plain_step(kv):
    c = Case(kv, [1, 64, 700, 3000, 0], 8, 1, 1, 4000, 0, seed=8, poison=False).to_gpu()
    got, _ = c.step()
    c.check(got)
    c.window = 0
    ref, _ = c.step()
    c.check(ref)
    # the same sums but for where the softmax's reference moves: each side is
    # within half the step of its weights' type twice, and of its BF16 output
    _, mass = c.reference()
    u = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    far = (got.double() - ref.double()).abs().cpu().numpy().reshape(mass.shape)
    assert (far <= (4 * u + 2.0 ** -7 + 1e-3) * mass + 1e-30).all()


def test_block_scales_that_are_one_scale_match_the_e4m3_cache():
    """The same numbers in both caches: the outputs agree within both kernels' roundings."""
    c = Case("e4m3", [900, 5, 64], 8, 2, 1, 200, 8, seed=9).to_gpu()
    got, _ = c.step()
    c.kv, P = "block", c.k.shape[0]
    c.scale = torch.empty((P, 2, 2, 4), device="cuda")
    c.scale[:, :, 0], c.scale[:, :, 1] = c.ks, c.vs
    again, _ = c.step()
    c.check(again)
    c.check(got)


@pytest.mark.parametrize("kv", KINDS)
def test_the_plan_leaves_out_exactly_the_hidden_tiles(kv):
    for n, W, S in ((1, 100, 5), (2, 640, 64), (1, 1, 129), (3, 5000, 0)):
        c = Case(kv, LENS, 4, 1, n, W, S, seed=60).to_gpu()
        ws = c.workspace(29)
        hd.hpc_decode_plan_win(c.sl, 1, c.bt.shape[1], 29, 2, ws.tmap, kv_dtype=DTYPE[kv], q_len=n,
                               window=W, sinks=S)
        torch.cuda.synchronize()
        got = ws.tmap.to_host()
        ref = oracle.assign_closed_form(ow.planned_lengths(LENS, c.bt.shape[1], n, W, S), 1, 29, 2)
        for name in ("total_tiles", "budget", "num_desc", "desc", "bin_ptr", "chunk_count",
                     "chunk_off"):
            assert got[name] == getattr(ref, name), name
        assert got["flags"] == 0


@pytest.mark.parametrize("kv", KINDS)
def test_plan_once_then_attention_on_several_layers(kv):
    """A map reused by two layers' attention calls, fused and with the separate combine."""
    c = Case(kv, LENS, 8, 2, 1, 150, 9, seed=61).to_gpu()
    ws = c.workspace()
    hd.hpc_decode_plan_win(c.sl, 2, c.bt.shape[1], ws.num_ctas, 2, ws.tmap, kv_dtype=DTYPE[kv],
                           window=150, sinks=9)
    args = (c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, c.bt, c.sl, 8, 2, 1, 150, 9, c.sm, ws.tmap,
            ws.part_o, ws.part_lse)
    outs = [torch.full((len(LENS), 1, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
            for _ in range(3)]
    hd.hpc_decode_attn_win(*args, outs[0], ws.unit_done)
    hd.hpc_decode_attn_win(*args, outs[1], ws.unit_done)
    hd.hpc_decode_attn_win(*args)
    hd.hpc_decode_combine_mq(ws.part_o, ws.part_lse, ws.tmap, len(LENS), 8, 2, 1, outs[2])
    torch.cuda.synchronize()
    for o in outs:
        c.check(o)
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    # another window, or none, is refused on this map
    with pytest.raises(hd.HpcError):
        hd.hpc_decode_attn_win(*args[:12], 151, 9, *args[14:], outs[0], ws.unit_done)
    with pytest.raises(hd.HpcError):
        hd.hpc_decode_attn_win(*args[:12], 0, 0, *args[14:], outs[0], ws.unit_done)


@pytest.mark.parametrize("kv", KINDS)
def test_more_requests_than_the_kernel_derives_itself(kv):
    rng = np.random.default_rng(5)
    for B in (65, 1030):  # above 64 the first bin is not walked, above 1024 not derived
        lens = [int(x) for x in rng.integers(0, 400, B)]
        c = Case(kv, lens, 4, 1, 1, 90, 3, seed=62).to_gpu()
        got, _ = c.step()
        c.check(got)


@pytest.mark.parametrize("kv", KINDS)
def test_long_context_and_many_bins(kv):
    c = Case(kv, [20000, 70, 9000], 8, 1, 1, 6000, 130, seed=63).to_gpu()
    for ctas in (0, 400, 1):
        got, _ = c.step(ctas=ctas)
        c.check(got)


@pytest.mark.parametrize("kv", KINDS)
def test_bad_lengths_and_pages_are_flagged(kv):
    c = Case(kv, [200, 300, 100], 4, 1, 1, 128, 0, seed=64, poison=False).to_gpu()
    ws = c.workspace()
    out = torch.zeros((3, 1, 4, 128), dtype=torch.bfloat16, device="cuda")

    def flags(bt, sl):
        hd.hpc_decode_step_win(c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, bt, sl, 4, 1, 1, 128, 0,
                               c.sm, ws.num_ctas, 2, ws.tmap, ws.part_o, ws.part_lse, out,
                               unit_done=ws.unit_done)
        torch.cuda.synchronize()
        return ws.tmap.to_host()["flags"]

    assert flags(c.bt, c.sl) == 0
    bad = c.bt.clone()
    bad[1, 0] = 999  # before the window of request 1 (172 .. 299): not looked at
    assert flags(bad, c.sl) == 0
    c.check(out)
    bad[1, 3] = 999
    assert flags(bad, c.sl) == 4
    long = c.sl.clone()
    long[0] = 64 * c.bt.shape[1] + 1
    assert flags(c.bt.clamp(min=0), long) == 1
    long[0] = -3
    assert flags(c.bt, long) == 1


def test_repeated_and_captured_launches_are_identical():
    c = Case("block", [3000, 64, 777, 1], 16, 2, 1, 512, 8, seed=65).to_gpu()
    first, ws = c.step()
    again, _ = c.step(ws=ws)
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    out = torch.zeros_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hd.hpc_decode_step_win(c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, c.bt, c.sl, 16, 2, 1, 512,
                               8, c.sm, ws.num_ctas, 2, ws.tmap, ws.part_o, ws.part_lse, out,
                               unit_done=ws.unit_done)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    # the lengths may change between replays: the plan is part of the graph
    c.sl.copy_(torch.tensor([100, 30, 64, 0], dtype=torch.int32))
    c.lens = [100, 30, 64, 0]
    c2 = Case("block", c.lens, 16, 2, 1, 512, 8, seed=65, poison=False).to_gpu()
    for name in ("k", "v", "scale", "bt", "q", "qs"):
        t, u = getattr(c, name), getattr(c2, name)
        t.view(-1).view(torch.uint8)[:u.numel() * u.element_size()] = u.view(-1).view(torch.uint8)
    c.bt.fill_(-1)
    c.bt[:, :c2.bt.shape[1]] = c2.bt
    g.replay()
    torch.cuda.synchronize()
    c2.check(out)


@pytest.mark.parametrize("kv", KINDS)
def test_two_captured_graphs_share_a_workspace(kv):
    """Steps over a window and over the whole context, captured with one workspace
    and replayed in turn on one stream: each leaves it as the other needs it."""
    c = Case(kv, [3000, 64, 777, 1], 16, 2, 1, 512, 8, seed=68, poison=False).to_gpu()
    ws = c.workspace()
    graphs, outs, eager = [], [], []
    for window, sinks in ((512, 8), (0, 0)):
        c.window, c.sinks = window, sinks
        eager.append(c.step(ws=ws)[0])
        out = torch.zeros_like(eager[-1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            hd.hpc_decode_step_win(c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, c.bt, c.sl, 16, 2, 1,
                                   window, sinks, c.sm, ws.num_ctas, 2, ws.tmap, ws.part_o,
                                   ws.part_lse, out, unit_done=ws.unit_done)
        graphs.append(g)
        outs.append(out)
    for k in (0, 1, 1, 0, 1, 0):
        outs[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[k].view(torch.int16), eager[k].view(torch.int16))
    assert int(torch.count_nonzero(ws.unit_done)) == 0


def test_two_streams_with_their_own_workspaces():
    cases = [Case(kv, LENS, 8, 1, 1, 200, 4, seed=66 + i).to_gpu()
             for i, kv in enumerate(("block", "bf16"))]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    ws = [c.workspace() for c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, w in zip(cases, streams, ws):
            out = torch.full((len(LENS), 1, 8, 128), float("nan"), dtype=torch.bfloat16,
                             device="cuda")
            s.wait_stream(torch.cuda.current_stream())
            hd.hpc_decode_step_win(c.q, c.qs, c.k, c.v, c.ks, c.vs, c.scale, c.bt, c.sl, 8, 1, 1,
                                   200, 4, c.sm, w.num_ctas, 2, w.tmap, w.part_o, w.part_lse, out,
                                   unit_done=w.unit_done, stream=s)
            outs.append((c, out))
    torch.cuda.synchronize()
    for c, o in outs:
        c.check(o)


# ------------------------------------------------------------------ prefill
def run_prefill(c, flags=None):
    shape = (len(c.lens), c.q_len, c.Hq, 128)
    out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    own = torch.zeros(1, dtype=torch.int32, device="cuda") if flags is None else flags
    hd.hpc_prefill_attn_win(c.q, c.k, c.v, c.bt, c.sl, c.Hq, c.Hkv, c.q_len, c.window, c.sinks,
                            c.sm, out, flags=own)
    torch.cuda.synchronize()
    if flags is None:
        assert int(own.item()) == 0
    return out


@pytest.mark.parametrize("win", WINDOWS + [(128, 0), (256, 128), (200, 129), (129, 0)])
@pytest.mark.parametrize("q_len", [1, 64, 129, 300])
def test_windowed_prefill(win, q_len):
    lens = [q_len, q_len + 1, q_len + 63, q_len + 400, q_len + 1000, max(q_len - 30, 0)]
    c = Case("bf16", lens, 2, 1, q_len, *win, seed=500).to_gpu()
    c.check(run_prefill(c))


@pytest.mark.parametrize("L", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 700])
@pytest.mark.parametrize("win", [(64, 4), (128, 128), (150, 0)])
def test_windowed_prefill_lengths(L, win):
    c = Case("bf16", [L], 2, 2, L, *win, seed=501).to_gpu()
    c.check(run_prefill(c))


@pytest.mark.parametrize("heads", [(8, 1), (4, 4), (6, 2), (16, 1), (32, 1)])
def test_windowed_prefill_heads(heads):
    c = Case("bf16", [300, 520], *heads, 260, 100, 10, seed=502).to_gpu()
    c.check(run_prefill(c))


@pytest.mark.parametrize("q_len,heads", [(700, 64), (520, 56), (256, 160)])
def test_windowed_prefill_of_several_rounds(q_len, heads):
    """More pairs of Q tiles than SMs (192, 168, 160): CTAs take several, and a
    short last round is cut into single Q tiles.  Sampled heads and rows."""
    c = Case("bf16", [q_len, q_len + 500], heads, heads // 8, q_len, 200, 70, seed=507).to_gpu()
    out = run_prefill(c)
    rows = sorted({0, 1, 127, 128, 129, 255, q_len - 1, q_len // 2} |
                  set(range(0, q_len, 37)))
    rows = [r for r in rows if r < q_len]
    hs = list(range(0, heads, 7)) + [heads - 1]
    ref = np.zeros((2, len(rows), len(hs), 128))
    mass = np.zeros(ref.shape)
    for r, L in enumerate(c.lens):
        see = ow.visible(L, q_len, 200, 70)[rows]
        for k, h in enumerate(hs):
            # (pages that were given back come as NaN: no row sees their tokens)
            K, V = (np.nan_to_num(ow.gather(x, c.table[r], L)[:, h // 8]) for x in (c.kf, c.vf))
            x = np.where(see, c.qf[r, rows, h] @ K.T * c.sm, -np.inf)
            e = np.exp(x - x.max(-1, keepdims=True))
            w = e / e.sum(-1, keepdims=True)
            ref[r, :, k], mass[r, :, k] = w @ V, w @ np.abs(V)
    check_attention(out[:, rows][:, :, hs], ref, mass, "bf16")
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("q_len", [300, 520, 700])
def test_windowed_prefill_of_several_rounds_of_an_odd_group(q_len):
    """Three query heads to a KV head: pairs are two Q tiles of a head (300 leaves
    the second of the last pair without rows), their last round cut into single
    tiles; requests shorter than q_len leave the first tile without tokens."""
    c = Case("bf16", [q_len, q_len + 200, q_len - 290], 63, 21, q_len, 90, 70, seed=508).to_gpu()
    c.check(run_prefill(c))


@pytest.mark.parametrize("heads", [(4, 2), (3, 1)])
@pytest.mark.parametrize("win", [(5000, 0), (4096, 130), (64, 2500), (6000, 1)])
def test_windowed_prefill_of_many_pages(heads, win):
    """More pages than a warp fetches entries of at once, sinks among them."""
    c = Case("bf16", [6000, 4200, 130], *heads, 200, *win, seed=509).to_gpu()
    c.check(run_prefill(c))


@pytest.mark.parametrize("kv", KINDS)
def test_requests_that_share_pages(kv):
    """A common prefix: the same pages in several rows of the block table, and one
    page twice in a row."""
    c = Case(kv, [700, 640, 300], 8, 2, 2, 260, 20, seed=510, poison=False)
    c.table[1, :6] = c.table[0, :6]
    c.table[2, :3] = c.table[0, :3]
    c.table[0, 9] = c.table[0, 8]
    c.to_gpu()
    got, _ = c.step()
    c.check(got)
    if kv == "bf16":
        c.check(run_prefill(c))


@pytest.mark.parametrize("kv", KINDS)
def test_pages_beyond_32_bit_offsets(kv):
    """The same pages at the end of a cache of more than 2^32 bytes."""
    c = Case(kv, [300, 700], 16, 8, 1, 200, 70, seed=512, poison=False).to_gpu()
    near, _ = c.step()
    if kv == "bf16":
        near_prefill = run_prefill(c)
    P = c.k.shape[0]
    N = P + (5 << 30) // (c.k[0].numel() * c.k.element_size())
    at = (N - 1 - torch.arange(P)).cuda()
    for name in ("k", "v", "scale"):
        t = getattr(c, name)
        if t is not None:
            far = torch.empty((N,) + t.shape[1:], dtype=t.dtype, device="cuda")
            far.view(torch.uint8)[at] = t.view(torch.uint8)
            setattr(c, name, far)
    c.bt = torch.where(c.bt >= 0, N - 1 - c.bt, c.bt)
    got, _ = c.step()
    assert torch.equal(got.view(torch.int16), near.view(torch.int16))
    if kv == "bf16":
        assert torch.equal(run_prefill(c).view(torch.int16), near_prefill.view(torch.int16))
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kv", KINDS)
def test_more_split_units_than_a_cta_keeps_for_the_end(kv):
    """Thousands of bins of one tile: a CTA completes more split units than it
    lists (16), and merges the others on the spot."""
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(65, 300, 1300)]
    c = Case(kv, lens, 8, 4, 1, 150, 3, seed=511).to_gpu()
    for fused in (True, False):
        got, ws = c.step(ctas=16000, floor=1, fused=fused)
        c.check(got)


def test_prefill_without_a_window_is_the_plain_call():
    w = Workload("pw", 2, 4, 2, seqlens=(300, 700), seed=503, q_len=290)
    b = make_batch(w, device="cuda", poison_tail=True)
    outs = [torch.zeros((2, 290, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    hd.hpc_prefill_attn(b.q, b.k_cache, b.v_cache, b.block_table, b.seqlens, 4, 2, 290,
                        w.sm_scale, outs[0])
    for o, win in zip(outs[1:], (0, 1000)):
        hd.hpc_prefill_attn_win(b.q, b.k_cache, b.v_cache, b.block_table, b.seqlens, 4, 2, 290,
                                win, 0, w.sm_scale, o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    # a window beyond every length is the same function, in a kernel whose
    # reference moves page by page: each is right by itself
    host = [x.double().cpu().numpy() for x in (b.q, b.k_cache, b.v_cache)]
    ref, mass = ow.attention(host[0].reshape(2, 290, 4, 128), host[1], host[2],
                             b.block_table.cpu().numpy(), (300, 700), 0, 0, w.sm_scale)
    for o in outs:
        check_attention(o, ref, mass, "bf16")


def test_prefill_flags():
    c = Case("bf16", [900, 600], 2, 1, 100, 128, 4, seed=504).to_gpu()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(run_prefill(c, flags))  # evicted pages hold bad entries: not looked at
    assert int(flags.item()) == 0
    keep = c.bt.clone()
    c.bt[0, 13] = 999
    run_prefill(c, flags)
    assert int(flags.item()) == 4
    flags.zero_()
    c.bt = keep
    c.sl[1] = -5
    run_prefill(c, flags)
    assert int(flags.item()) == 1


def test_prefill_is_deterministic_and_captures():
    c = Case("bf16", [2000], 8, 2, 1500, 300, 70, seed=505).to_gpu()
    a = run_prefill(c)
    out = torch.zeros_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hd.hpc_prefill_attn_win(c.q, c.k, c.v, c.bt, c.sl, 8, 2, 1500, 300, 70, c.sm, out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), out.view(torch.int16))
    c.check(a)


def test_decode_and_prefill_agree_on_the_last_tokens():
    """The same queries through both forms (BF16 cache), each against the oracle."""
    c = Case("bf16", [1000, 300, 77], 8, 1, 2, 256, 20, seed=506).to_gpu()
    got, _ = c.step()
    c.check(got)
    c.check(run_prefill(c))
