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


@pytest.mark.parametrize("kv", KINDS)
def test_no_groups_and_empty_batches(kv):
    lens = [300, 0, 64, 1]
    c = Shared(kv, lens, [0], [], 8, 2, 2, seed=5).to_gpu()
    got, ws = c.step()
    c.check_plan(ws)
    c.check(got)
    # nothing to share: groups of one, of none, of no pages, of members that are too short
    c = Shared(kv, lens, [0, 1, 1, 3, 4], [4, 1, 0, 3], 8, 2, 2, seed=6).to_gpu()
    got, ws = c.step()
    c.check_plan(ws)
    c.check(got)
    assert ws.head_ctas() == 0
    none = Shared(kv, [0] * 5, [0, 5], [0], 8, 2, 1, seed=7).to_gpu()
    got, ws = none.step()
    assert not got.float().abs().sum()
    e = c.q[:0]
    hd.hpc_decode_step_shared(e, None if c.qs is None else c.qs[:0], c.k, c.v, c.ks, c.vs, c.scale,
                              c.bt[:0], c.sl[:0], torch.zeros(1, dtype=torch.int32, device="cuda"),
                              c.sl[:0], 8, 2, 2, c.sm, 2,
                              hd.SharedWorkspace(0, 8, 2, 0, kv_dtype=ws.kv_dtype, q_len=2), c.out()[:0])


def test_bad_groups_and_lengths_are_flagged():
    c = Shared("bf16", wide(12, 2, 1, 3), [0, 12], [2], 8, 1, 1, seed=8).to_gpu()
    ref, mass = c.reference()
    for starts, pages in (([3, 2], [2]), ([0, 13], [2]), ([-1, 4], [1]), ([0, 12], [-1]),
                          ([0, 12], [1000])):
        c.starts, c.pages = starts, pages
        got, ws = c.step(flags=hd.binding.HPC_FLAG_BAD_SEQLEN)
        assert ws.head_ctas() == 0  # nothing is shared, and everything computed
        c.check(got)
    c.starts, c.pages = [0, 12], [2]
    c.sl[2] = -5
    c.sl[4] = 10 ** 9  # taken as all of its row
    got, ws = c.step(flags=hd.binding.HPC_FLAG_BAD_SEQLEN | hd.binding.HPC_FLAG_BAD_PAGE)
    assert not got[2].float().abs().sum()
    keep = [r for r in range(12) if r not in (2, 4)]
    from _shared import check_shared
    check_shared(got[keep], ref[keep], mass[keep], "bf16")


@pytest.mark.parametrize("kv", KINDS)
def test_bad_pages_are_flagged_and_not_read(kv):
    c = Shared(kv, wide(10, 3, 1, 4), [0, 10], [3], 16, 2, 1, seed=9).to_gpu()
    c.bt[0, 1] = c.k.shape[0] + 1000  # of the shared ones
    c.bt[7, 3] = -3                   # of a tail
    got, _ = c.step(flags=hd.binding.HPC_FLAG_BAD_PAGE)
    # the prefix is looked up in the first sharing request's row only
    c.bt[0, 1] = int(c.table[0, 1])
    c.bt[7, 3] = int(c.table[7, 3])
    c.bt[5, 0] = -9
    got, _ = c.step()
    c.check(got)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("sm", [-0.05, 0.0, 0.3])
def test_score_scales_of_any_sign(kv, sm):
    c = Shared(kv, wide(18, 3, 1, 5), [0, 18], [3], 16, 2, 1, seed=10).to_gpu()
    c.sm = sm
    if kv != "bf16":  # and queries whose scale turns them round
        c.qs[::3] *= -1
        c.qf[::3] *= -1
    got, _ = c.step()
    c.check(got)


def test_block_scales_of_any_size():
    """K scales of either sign, V scales from 2^-100 to 2^100 and zero, in the shared pages and
    behind them."""
    c = Shared("block", wide(20, 3, 1, 6), [0, 20], [3], 8, 1, 1, seed=11, poison=False)
    rng = np.random.default_rng(5)
    s = c.scale.numpy()
    s[:, :, 0] *= rng.uniform(-1.0, 1.0, s[:, :, 0].shape)
    s[:, :, 1] = np.exp2(rng.uniform(-100, 100, s[:, :, 1].shape))
    s[:, :, 1][rng.random(s[:, :, 1].shape) < 0.2] = 0.0
    from oracle import block_cache as bc
    c.kf, c.vf = (bc.values(x.view(torch.uint8).numpy(), s, i) for i, x in enumerate((c.k, c.v)))
    got, _ = c.to_gpu().step()
    c.check(got)


@pytest.mark.parametrize("kv", KINDS)
def test_scores_that_climb(kv):
    """Each page's scores stand far above the last one's: the reference moves at every page,
    and what was summed before nearly vanishes."""
    c = Shared(kv, wide(20, 12, 1, 7), [0, 20], [12], 8, 1, 1, seed=12, poison=False)
    rows = c.table[0]
    x = torch.zeros(c.k.shape, dtype=torch.float32)
    x[..., 1:] = 0.01 * torch.randn(x[..., 1:].shape, generator=torch.Generator().manual_seed(1))
    for t in range(12):
        x[int(rows[t]), :, :, 0] = 20.0 * t
    q = torch.zeros(c.q.shape, dtype=torch.float32)
    q[..., 0], q[..., 5] = 8.0, 1.0
    if kv == "bf16":
        c.k, c.q = x.bfloat16(), q.bfloat16()
        c.kf, c.qf = c.k.double().numpy(), c.q.double().numpy()
    else:
        E4M3 = torch.float8_e4m3fn
        c.ks = 0.5
        c.k, c.q = (x * 2).clamp(-448, 448).to(E4M3), q.to(E4M3)
        c.qs = torch.ones(c.qs.shape)
        c.kf, c.qf = c.k.float().double().numpy() * 0.5, c.q.float().double().numpy()
        if c.scale is not None:
            c.scale[:, :, 0] = 0.5
    got, _ = c.to_gpu().step(ctas=2)
    c.check(got)


def test_a_plan_serves_many_layers_and_graphs_share_a_workspace():
    """Planned once, several layers' attention; two captured steps on one workspace, replayed
    in turn, with other lengths, groups and pages in between; on streams of their own."""
    a = Shared("bf16", wide(24, 3, 1, 8), [0, 14, 24], [3, 2], 8, 1, 1, seed=13).to_gpu()
    b = Shared("bf16", wide(24, 4, 1, 9), [0, 24, 24], [4, 7], 8, 1, 1, seed=14).to_gpu()
    ws = a.workspace()
    two = {}
    for name, c in (("a", a), ("b", b)):
        c.dev = c.groups()
        c.o = [c.out(), c.out()]
        c.q2 = (c.q.float() * 0.5).bfloat16()
    torch.cuda.synchronize()

    def layers(c):
        starts, pages = c.dev
        hd.hpc_decode_plan_shared(c.sl, starts, pages, 8, 1, 1, c.bt.shape[1], 2, ws)
        for q, o in ((c.q, c.o[0]), (c.q2, c.o[1])):
            hd.hpc_decode_attn_shared(q, None, c.k, c.v, 1.0, 1.0, None, c.bt, c.sl, 8, 1, 1, c.sm,
                                      ws, o)

    stream = torch.cuda.Stream()
    for name, c in (("a", a), ("b", b)):
        with torch.cuda.stream(stream):
            layers(c)  # (a first call prepares the kernel)
        torch.cuda.synchronize()
        two[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(two[name], stream=stream):
            layers(c)
        torch.cuda.synchronize()
    for name in ("a", "b", "a", "b"):
        c = {"a": a, "b": b}[name]
        for o in c.o:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        two[name].replay()
        torch.cuda.synchronize()
        assert ws.flags == 0
        c.check(c.o[0])
        c.qf = c.q2.double().cpu().numpy()
        c.check(c.o[1])
        c.qf = c.q.double().cpu().numpy()
    # other lengths in the captured step: all but three members are too short to share
    a.lens = [min(n, 100) if r % 4 else n for r, n in enumerate(a.lens)]
    a.sl.copy_(torch.tensor(a.lens, dtype=torch.int32))
    two["a"].replay()
    torch.cuda.synchronize()
    a.check(a.o[0])


def test_offsets_past_32_bits():
    """Pages whose bytes lie beyond 2^32 in each cache."""
    P, B, Hq, Hkv = 40000, 10, 64, 8  # 128 KB a page: 5.2 GB of K and of V
    lens = [64 * 5 + 3 * r for r in range(B)]
    c = Shared("bf16", lens, [0, B], [5], Hq, Hkv, 1, seed=15)
    used = c.k.shape[0]
    big = [torch.zeros((P, 64, Hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, x in zip(big, (c.k, c.v)):
        t[P - used:] = x.cuda()
    c.to_gpu()
    c.k, c.v = big
    c.bt[c.bt >= 0] += P - used
    got, _ = c.step()
    c.check(got)


def test_results_repeat_bit_for_bit():
    for kv in KINDS:
        c = Shared(kv, wide(40, 6, 1, 10), [0, 40], [6], 16, 2, 1, seed=16).to_gpu()
        first, ws = c.step()
        for _ in range(3):
            again, _ = c.step(ws=ws)
            assert torch.equal(first, again)


@pytest.mark.parametrize("kv", KINDS)
def test_not_a_number_reaches_the_rows_that_see_it_and_no_others(kv):
    """NaN in a key of a shared page: all that the group's sharing rows get of that KV head is
    NaN, whatever the other partials are; all other rows keep their bits."""
    lens = wide(20, 40, 1, 11) + wide(9, 3, 1, 12) + [200]
    c = Shared(kv, lens, [0, 20, 29], [40, 3], 16, 2, 1, seed=17).to_gpu()
    clean, ws = c.step()
    page = c.table[0, 17]
    if kv == "bf16":
        c.k[page, 5, 1, 7] = float("nan")
    else:
        c.k.view(torch.uint8)[page, 5, 1, 7] = 0x7F
    got, _ = c.step(ws=ws)
    hit = torch.zeros(len(lens), 1, 16, dtype=torch.bool)
    for r, (g, _) in c.lead.items():
        hit[r, :, 8:] |= g == 0
    nan = got.isnan().cpu()
    assert torch.equal(nan.all(-1), hit) and torch.equal(nan.any(-1), hit)
    assert torch.equal(got.cpu()[~hit], clean.cpu()[~hit])


def test_the_largest_batch():
    """8192 requests in 4096 groups of two; a batch smaller than its workspace; as many
    CTAs as a plan may have, many more than the GPU has SMs."""
    B = 8192
    lens = [64 + (7 * r) % 90 for r in range(B)]
    c = Shared("bf16", lens, list(range(0, B + 1, 2)), [1] * (B // 2), 1, 1, 1, seed=18).to_gpu()
    got, ws = c.step()
    c.check_plan(ws)
    c.check(got)
    small = Shared("bf16", wide(20, 3, 1, 13), [0, 20], [3], 1, 1, 1, seed=19).to_gpu()
    small.n = 1
    got, _ = small.step(ws=ws)
    small.check_plan(ws)
    small.check(got)
    for kv in KINDS:
        many = Shared(kv, wide(30, 50, 1, 14), [0, 30], [50], 8, 2, 1, seed=20).to_gpu()
        for ctas in (500, 65536):
            got, ws = many.step(ctas=ctas, floor=1)
            many.check_plan(ws)
            many.check(got)


def test_two_streams_at_once():
    """Steps on two streams, each with a workspace of its own."""
    cases = [Shared(kv, wide(24, 30, 1, 15 + i), [0, 24], [30], 16, 2, 1, seed=21 + i).to_gpu()
             for i, kv in enumerate(("bf16", "e4m3"))]
    for c in cases:
        c.ws, c.o, c.dev = c.workspace(), [c.out() for _ in range(20)], c.groups()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for c, s in zip(cases, streams):
            hd.hpc_decode_step_shared(c.q, c.qs, c.k, c.v, c.ks, c.vs, None, c.bt, c.sl, *c.dev, 16, 2,
                                      1, c.sm, 2, c.ws, c.o[i], stream=s)
    torch.cuda.synchronize()
    for c in cases:
        assert c.ws.flags == 0
        c.check(c.o[0])
        assert all(torch.equal(o, c.o[0]) for o in c.o)
