"""The block-scaled 8-bit cache: the prologue that writes it and its read-back
against the fp64 oracle, and a run of a prompt in chunks with decode steps."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from _blocks import E4M3, Case, Prologue, check_attention
from oracle import block_cache as bc
from oracle import rope_norm as rn
from oracle import window as ow

pytestmark = pytest.mark.gpu

# fp32 error of the norm and the rotation, relative to the row's largest
# value: the mean of 128 squares, rsqrt, three products and the rotation's
# two-term sum, each 2^-24, and an angle error of 1e-6 rad (positions here are
# below 2^15) come to less than 4e-6
EPS = 4e-6


def tokens_of(spans):
    """[(request, position), ...] of spans (request, first, count)."""
    return [(r, p) for r, a, n in spans for p in range(a, a + n)]


def check_queries(pro, q):
    got = pro.q[:pro.N].float().cpu().double().numpy()
    big = np.abs(q).max(-1, keepdims=True)
    if not pro.q8:  # BF16: half a step of the value, and the fp32 error
        assert (np.abs(got - q) <= 2.0 ** -8 * np.abs(q) + EPS * big).all()
        return
    s = pro.qs[:pro.N].cpu().double().numpy()[..., None]
    want = np.where(big > 0, big / 448, 1.0)
    assert (np.abs(s - want) <= 2 * EPS * want).all()
    # E4M3: half a step (2^-4 of the value, 2^-10 of the scale below the normal range)
    assert (np.abs(got * s - q) <= 2.0 ** -4 * np.abs(q) + 2.0 ** -10 * s + 2 * EPS * big).all()


def check_cache(pro, k, v):
    """Codes, scales and every slot that was not written."""
    (kc, ks, runs, flags), (vc, vs, _, _) = pro.oracle_write(k, v)
    assert int(pro.flags.item()) == flags
    got_s = pro.scale.cpu().numpy()
    got_k, got_v = (t.view(torch.uint8).cpu().numpy() for t in (pro.k, pro.v))
    # V is BF16 input over a power of two: every code, every scale exact
    assert np.array_equal(got_s[:, :, 1].astype(np.float64), vs)
    assert np.array_equal(got_v, vc)
    # K: a run's maximum is known to EPS, so its scale may differ where it lies
    # that near a border; then codes differ, but not what they stand for
    touched = np.zeros(got_k.shape[:2], dtype=bool)
    for pg, b, toks in runs:
        touched[pg, 16 * b:16 * b + 16] = True
        off = np.array([int(pro.pos[t]) % 16 for t in toks])
        for h in range(pro.Hkv):
            s = float(got_s[pg, h, 0, b])
            fresh = 0 in off
            old = None if fresh else float(pro.scale0[pg, h, 0, b])
            near = {bc.run_scale(k[toks, h] * f, old) for f in (1 - EPS, 1.0, 1 + EPS)}
            assert s in near
            val = rn.e4m3_decode(got_k[pg, 16 * b:16 * b + 16, h]) * s
            last = {int(o): t for t, o in zip(toks, off)}  # the later token stays
            for o, t in last.items():
                y, big = k[t, h], np.abs(k[t, h]).max()
                tol = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * s + EPS * big
                assert (np.abs(val[o] - y) <= tol).all()
            rest = [o for o in range(16) if o not in last]
            if s == ks[pg, h, b]:
                assert np.array_equal(got_k[pg, 16 * b:16 * b + 16, h][rest],
                                      kc[pg, 16 * b:16 * b + 16, h][rest])
    assert np.array_equal(got_k[~touched], pro.codes0[0][~touched])
    # codes that are not the oracle's can only sit next to a rounding border
    assert (got_k != kc).mean() <= 1e-3
    other = np.ones(got_s.shape[:1] + (4,), dtype=bool)
    for pg, b, _ in runs:
        other[pg, b] = False
    o = np.broadcast_to(other[:, None, None, :], got_s.shape)
    assert np.array_equal(got_s[o], pro.scale0[o])


def check_write(pro):
    q, k, v = pro.exact_rows()
    check_queries(pro, q)
    check_cache(pro, k, v)


SPANS = {
    "one": [(0, 0, 1)],
    "decode": [(r, p, 1) for r, p in enumerate((0, 1, 15, 16, 17, 63, 64, 100, 127))],
    "prompt": [(0, 0, 130)],
    "ragged": [(0, 3, 5), (1, 0, 33), (2, 15, 2), (3, 60, 70), (4, 31, 1), (5, 16, 16)],
    "draft": [(r, p, 3) for r, p in enumerate((0, 14, 15, 62, 90))],
}


@pytest.mark.parametrize("spans", list(SPANS))
@pytest.mark.parametrize("heads", [(8, 1), (2, 2), (12, 4), (9, 3)])
@pytest.mark.parametrize("q8", [True, False])
def test_write(spans, heads, q8):
    t = tokens_of(SPANS[spans])
    pro = Prologue(t, *heads, B=9, max_pages=3, seed=len(t) + heads[0], q8=q8).run()
    check_write(pro)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("norm_first", [True, False])
def test_write_orders_and_layouts(layout, norm_first):
    t = tokens_of(SPANS["ragged"])
    freq = torch.empty(64, dtype=torch.float64, device="cuda")
    hd.hpc_rope_frequencies(1e6, freq)
    for f in (None, freq):
        pro = Prologue(t, 8, 2, 9, 3, seed=77, layout=layout, norm_first=norm_first, pad=24)
        check_write(pro.run(freq=f))


def test_write_many_tokens():
    """Enough tokens for the larger chunks a CTA owns (2, 4 and 8 of them)."""
    for n, seed in ((700, 1), (1900, 2), (2700, 3), (5200, 4)):
        t = tokens_of([(0, 5, n // 2), (1, 0, n - n // 2 - 1), (2, 9, 1)])
        pro = Prologue(t, 1, 1, 3, 64, seed=seed).run()
        check_write(pro)


def test_appending_token_by_token_and_growth():
    """A block written by sixteen calls, sizes going up and down: the oracle's
    codes and scales after each (V: exactly)."""
    rng = np.random.default_rng(8)
    pro = Prologue([(0, 16), (1, 48)], 4, 1, 2, 2, seed=9)
    for step in range(16):
        pro.pos = np.array([16 + step, 48 + step], dtype=np.int32)
        grow = 2.0 ** float(rng.integers(-12, 13))
        rows = (torch.randn((2, 6, 128)) * grow).bfloat16()
        pro.qkv_host, pro.full = rows, rows.view(2, -1)
        pro.run()
        check_write(pro)
        pro.codes0 = [t.view(torch.uint8).cpu().numpy().copy() for t in (pro.k, pro.v)]
        pro.scale0 = pro.scale.cpu().numpy().copy()


def test_old_scales_that_are_none():
    """An append to a block whose scale is NaN, infinite, zero or negative, and one
    that is no power of two and stays."""
    t = [(r, 20 + r) for r in range(5)]
    pro = Prologue(t, 2, 1, 5, 1, seed=10)
    for r, s in enumerate((np.nan, np.inf, 0.0, -1.0, 3.7)):
        pro.scale0[pro.table[r, 0], :, :, 1] = s
    check_write(pro.run())


def test_zero_rows_and_non_finite_values():
    pro = Prologue(tokens_of([(0, 0, 4), (1, 3, 2)]), 2, 1, 2, 1, seed=11)
    rows = pro.qkv_host
    rows[1] = 0.0  # a token of zeros
    rows[4:, 3] = 0.0  # request 1: V all zero, appended
    rows[2, 3, 5], rows[2, 3, 6], rows[3, 3, 0] = float("inf"), float("nan"), -float("inf")
    pro.full = rows.view(6, -1)
    pro.run()
    q, k, v = pro.exact_rows()
    check_cache_v = pro.oracle_write(k, v)[1]
    got = pro.v.view(torch.uint8).cpu().numpy()
    want = check_cache_v[0]
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan)
    assert np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(pro.scale.cpu().numpy()[:, :, 1].astype(np.float64), check_cache_v[1])
    check_queries(pro, q)


def test_the_same_position_twice_and_too_many_tokens():
    # position 2 three times (the last stays), in rows held by both half-warps
    pro = Prologue([(0, 1), (0, 2), (0, 3), (0, 2), (0, 2), (0, 4)], 2, 1, 1, 1, seed=12).run()
    check_write(pro)
    # 18 tokens of one block: the first 16 count, the rest are refused with a flag
    pro = Prologue(tokens_of([(0, 0, 16)]) + [(0, 3), (0, 4), (0, 16)], 2, 1, 1, 1, seed=13).run()
    assert int(pro.flags.item()) == 1
    check_write(pro)


def test_bad_tokens_write_no_slot_but_get_their_query():
    t = [(0, 5), (7, 0), (-1, 3), (1, -1), (1, 128), (1, 70), (2, 64)]
    pro = Prologue(t, 4, 2, 3, 2, seed=14)
    pro.table[1, 1], pro.table[2, 1] = -1, 10 ** 6
    # RoPE of a token outside the cache's range turns by its position as given
    pro.run()
    assert int(pro.flags.item()) == 5
    check_write(pro)


def test_no_tokens_and_token_t_is_request_t():
    pro = Prologue([(0, 5)], 4, 2, 3, 2, seed=15)
    hd.hpc_rope_norm_block(pro.full.cuda()[:0], pro.wq.cuda(), pro.wk.cuda(),
                           torch.zeros(0, dtype=torch.int32, device="cuda"), None, 4, 2,
                           torch.from_numpy(pro.table).cuda(),
                           *(torch.from_numpy(c).cuda().view(E4M3) for c in pro.codes0),
                           torch.from_numpy(pro.scale0).cuda(),
                           torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    pro = Prologue([(0, 5), (1, 33), (2, 64)], 4, 2, 3, 2, seed=16).run()
    k, v, s = (t.view(torch.uint8).clone() for t in (pro.k, pro.v, pro.scale))
    k2, v2 = (torch.from_numpy(c.copy()).cuda().view(E4M3) for c in pro.codes0)
    s2 = torch.from_numpy(pro.scale0.copy()).cuda()
    hd.hpc_rope_norm_block(pro.full.cuda(), pro.wq.cuda(), pro.wk.cuda(),
                           torch.from_numpy(pro.pos).cuda(), None, 4, 2,
                           torch.from_numpy(pro.table).cuda(), k2, v2, s2, pro.q, pro.qs)
    torch.cuda.synchronize()
    assert torch.equal(k, k2.view(torch.uint8)) and torch.equal(v, v2.view(torch.uint8))
    assert torch.equal(s, s2.view(torch.uint8))


def test_write_and_read_of_pages_beyond_32_bit_offsets():
    """The same tokens into the end of a cache of more than 2^32 bytes."""
    pro = Prologue([(r, p) for r in range(2) for p in range(30, 70)], 16, 8, 2, 2, seed=18).run()
    P = pro.P
    N = P + (5 << 30) // (64 * 8 * 128)
    at = (N - 1 - torch.arange(P)).cuda()
    far = []
    for host in (*pro.codes0, pro.scale0):
        t = torch.from_numpy(host.copy()).cuda()
        big = torch.empty((N,) + t.shape[1:], dtype=t.dtype, device="cuda")
        big[at] = t
        far.append(big)
    k, v, s = far[0].view(E4M3), far[1].view(E4M3), far[2]
    table = torch.from_numpy(N - 1 - pro.table).cuda()
    q, qs = torch.zeros_like(pro.q), torch.zeros_like(pro.qs)
    hd.hpc_rope_norm_block(pro.full.cuda(), pro.wq.cuda(), pro.wk.cuda(),
                           torch.from_numpy(pro.pos).cuda(), torch.from_numpy(pro.req).cuda(), 16,
                           8, table, k, v, s, q, qs)
    for big, small in ((k, pro.k), (v, pro.v)):
        assert torch.equal(big.view(torch.uint8)[at], small.view(torch.uint8))
    assert torch.equal(s[at], pro.scale)
    assert torch.equal(q.view(torch.uint8), pro.q.view(torch.uint8)) and torch.equal(qs, pro.qs)
    lens = torch.tensor([70, 70], dtype=torch.int32, device="cuda")
    outs = []
    for kc, vc, sc, bt in ((k, v, s, table),
                           (pro.k, pro.v, pro.scale, torch.from_numpy(pro.table).cuda())):
        out = [torch.zeros((4, 64, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        hd.hpc_kv_read_block(kc, vc, sc, bt, None, lens, 8, *out,
                             torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2))
        outs.append(out)
    for i in range(2):
        assert torch.equal(outs[0][i].view(torch.int16), outs[1][i].view(torch.int16))
    del far, k, v, s
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ read back
def run_read(codes, scale, table, starts, lens, Hkv, out_pages, out_table, fill=-77.0):
    k, v = (torch.from_numpy(c).cuda().view(E4M3) for c in codes)
    out = [torch.full((out_pages, 64, Hkv, 128), fill, dtype=torch.bfloat16, device="cuda")
           for _ in range(2)]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    hd.hpc_kv_read_block(k, v, torch.from_numpy(scale).cuda(), torch.from_numpy(table).cuda(),
                         None if starts is None else torch.tensor(starts, **i32),
                         torch.tensor(lens, **i32), Hkv, *out, torch.from_numpy(out_table).cuda(),
                         flags)
    torch.cuda.synchronize()
    return out, int(flags.item())


@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("pow2", [True, False])
def test_read_back(Hkv, pow2):
    rng = np.random.default_rng(20 + Hkv)
    starts, lens = [0, 5, 64, 70, 17, 0, 130, 200], [1, 64, 65, 200, 17, 0, 129, 400]
    B, mp, omp = len(lens), 8, 7
    P, OP = B * mp, B * omp
    table = rng.permutation(P).reshape(B, mp).astype(np.int32)
    out_table = rng.permutation(OP).reshape(B, omp).astype(np.int32)
    codes = [rng.integers(0, 255, (P, 64, Hkv, 128)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[c == 0xFF] = 0x12
        c[(c & 0x7F) == 0x7F] = 0x33
    e = rng.uniform(-20, 20, (P, Hkv, 2, 4))
    scale = np.exp2(np.rint(e) if pow2 else e).astype(np.float32)
    out, flags = run_read(codes, scale, table, starts, lens, Hkv, OP, out_table)
    assert flags == 0
    for i in range(2):
        # fp32 product, rounded to BF16: exact for powers of two, else two
        # roundings (2^-24 and 2^-8 of the value)
        val = bc.values(codes[i], scale, i)
        want = np.full((OP, 64, Hkv, 128), -77.0)
        for r in range(B):
            for t in range(starts[r], lens[r]):
                want[out_table[r, t // 64], t % 64] = val[table[r, t // 64], t % 64]
        got = out[i].double().cpu().numpy()
        tol = 0.0 if pow2 else 2.0 ** -8 + 2.0 ** -23
        assert (np.abs(got - want) <= tol * np.abs(want)).all()


def test_read_back_flags_and_large_batches():
    rng = np.random.default_rng(30)
    codes = [rng.integers(0, 0x7E, (4, 64, 1, 128)).astype(np.uint8) for _ in range(2)]
    scale = np.ones((4, 1, 2, 4), dtype=np.float32)
    table = np.array([[0, 1], [2, 9]], dtype=np.int32)
    same = np.array([[0, 1], [2, 3]], dtype=np.int32)
    out, flags = run_read(codes, scale, table, None, [128, 128], 1, 4, same)
    assert flags == 4  # page 9 is outside the cache: left out
    assert (out[0][3] == -77).all() and not (out[0][2] == -77).any()
    assert run_read(codes, scale, same, None, [129, 5], 1, 4, same)[1] == 1
    assert run_read(codes, scale, same, [-1, 0], [12, 5], 1, 4, same)[1] == 1
    assert run_read(codes, scale, same, None, [-4, 5], 1, 4, same)[1] == 1
    assert run_read(codes, scale, same, [500, 6], [100, 5], 1, 4, same)[1] == 0  # empty ranges
    bad = same.copy()
    bad[0, 1] = 4
    assert run_read(codes, scale, same, None, [128, 1], 1, 4, bad)[1] == 4
    # more requests than the prefix sum's small shared memory holds
    B = 12000
    table = (np.arange(B, dtype=np.int32) % 4)[:, None].copy()
    out_table = np.full((B, 1), -1, dtype=np.int32)
    out_table[::3000, 0] = np.arange(4)
    lens = np.where(np.arange(B) % 3000 == 0, 64, 0)
    out, flags = run_read(codes, scale, table, None, lens.tolist(), 1, 4, out_table)
    assert flags == 0
    for i in range(4):
        want = bc.values(codes[0], scale, 0)[table[3000 * i, 0]]
        assert np.array_equal(out[0][i].double().cpu().numpy(), want)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 10)])
def test_a_prompt_in_chunks_then_decode_steps(window, sinks):
    """A serving run of one layer: the prompt in two chunks (write, read the cache
    back as BF16 pages, windowed prefill attention over them), then decode steps
    with a draft token (write, attention over the 8-bit cache), on one stream with
    nothing waited for in between.  Each attention is compared with the oracle on
    the cache's contents at that point."""
    Hq, Hkv, B, mp = 8, 2, 3, 6
    chunks = [[100, 64, 7], [60, 77, 130]]
    gen = torch.Generator().manual_seed(50)
    dev = dict(device="cuda")
    P = B * mp
    table = torch.randperm(P, generator=gen).int().view(B, mp).cuda()
    k8, v8 = (torch.zeros((P, 64, Hkv, 128), dtype=torch.uint8, **dev).view(E4M3) for _ in "kv")
    scale = torch.full((P, Hkv, 2, 4), float("nan"), **dev)
    kb, vb = (torch.zeros((P, 64, Hkv, 128), dtype=torch.bfloat16, **dev) for _ in "kv")
    w = (1 + torch.randn(128, generator=gen) / 4).bfloat16().cuda()
    freq = torch.empty(64, dtype=torch.float64, **dev)
    hd.hpc_rope_frequencies(1e6, freq)
    flags = torch.zeros(1, dtype=torch.int32, **dev)
    sm, done = 128 ** -0.5, [0] * B
    checks = []

    def write(counts, q8):
        t = tokens_of([(r, done[r], counts[r]) for r in range(B)])
        qkv = torch.randn((len(t), (Hq + 2 * Hkv) * 128), generator=gen).bfloat16().cuda()
        q = torch.zeros((len(t), Hq, 128), dtype=E4M3 if q8 else torch.bfloat16, **dev)
        qs = torch.zeros((len(t), Hq), **dev) if q8 else None
        req, pos = (torch.tensor([x[i] for x in t], dtype=torch.int32).cuda() for i in (0, 1))
        hd.hpc_rope_norm_block(qkv, w, w, pos, req, Hq, Hkv, table, k8, v8, scale, q, qs, flags,
                               freq=freq)
        for r in range(B):
            done[r] += counts[r]
        return q, qs

    def snapshot(kind, q, qs, out, n, reqs, lens):
        checks.append((kind, q, qs, out, n, reqs, list(lens), k8.view(torch.uint8).clone(),
                       v8.view(torch.uint8).clone(), scale.clone()))

    for counts in chunks:
        before = list(done)
        q, _ = write(counts, False)
        sl = torch.tensor(done, dtype=torch.int32).cuda()
        hd.hpc_kv_read_block(k8, v8, scale, table, torch.tensor(before, dtype=torch.int32).cuda(),
                             sl, Hkv, kb, vb, table, flags)
        at = 0
        for r in range(B):  # q_len differs by request: one prefill call each
            n = counts[r]
            qr = q[at:at + n].view(1, n, Hq, 128)
            out = torch.zeros_like(qr)
            hd.hpc_prefill_attn_win(qr, kb, vb, table[r:r + 1], sl[r:r + 1], Hq, Hkv, n, window,
                                    sinks, sm, out, flags)
            snapshot("bf16", qr, None, out, n, [r], [done[r]])
            at += n
    ws = hd.Workspace(B, Hq, Hkv, kv_dtype=hd.HPC_KV_E4M3_BLOCK, q_len=2)
    for _ in range(9):
        q, qs = write([2] * B, True)
        sl = torch.tensor(done, dtype=torch.int32).cuda()
        out = torch.zeros((B, 2, Hq, 128), dtype=torch.bfloat16, **dev)
        hd.hpc_decode_step_win(q, qs, k8, v8, 1.0, 1.0, scale, table, sl, Hq, Hkv, 2, window,
                               sinks, sm, ws.num_ctas, 2, ws.tmap, ws.part_o, ws.part_lse, out,
                               unit_done=ws.unit_done)
        snapshot("block", q, qs, out, 2, list(range(B)), done)
    torch.cuda.synchronize()
    assert int(flags.item()) == 0
    tab = table.cpu().numpy()
    for kind, q, qs, out, n, reqs, lens, kc, vc, sc in checks:
        s = np.nan_to_num(sc.cpu().numpy(), nan=0.0)  # blocks nothing has been written to
        kf, vf = (bc.values(c.cpu().numpy(), s, i) for i, c in enumerate((kc, vc)))
        qf = q.float().double().cpu().numpy().reshape(len(reqs), n, Hq, 128)
        if qs is not None:
            qf = qf * qs.double().cpu().numpy().reshape(len(reqs), n, Hq)[..., None]
        ref, mass = ow.attention(qf, kf, vf, tab[reqs], lens, window, sinks, sm)
        check_attention(out, ref, mass, kind)
