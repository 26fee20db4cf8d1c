"""Decode attention over shared prefixes at the ends of its inputs' ranges: V scales, values
that are not finite, bad table entries.  What can be is checked against the fp64 oracle."""

import numpy as np
import pytest
import torch

from _blocks import Case, check_attention
from _shared import Shared, check_shared
from oracle import block_cache as bc

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "block"]
E4M3 = torch.float8_e4m3fn


def set_keys(c, value_of_page, other):
    """Keys and queries of which only dim 0 is not zero: the score of a token is 8 times its
    page's value (table entry t of the shared pages: value_of_page[t], the other pages: other),
    times sm_scale."""
    x = torch.full((c.k.shape[0],), float(other))
    for t, v in enumerate(value_of_page):
        x[int(c.table[0, t])] = v
    k = torch.zeros(c.k.shape, dtype=torch.float32)
    k[..., 0] = x[:, None, None]
    q = torch.zeros(c.q.shape, dtype=torch.float32)
    q[..., 0] = 8.0
    if c.kv == "bf16":
        c.k, c.q = k.bfloat16(), q.bfloat16()
        c.kf, c.qf = c.k.double().numpy(), c.q.double().numpy()
        return
    c.k, c.q, c.ks = k.to(E4M3), q.to(E4M3), 1.0
    c.qs = torch.ones(c.qs.shape)
    c.kf, c.qf = c.k.float().double().numpy(), c.q.float().double().numpy()
    if c.scale is not None:
        c.scale[:, :, 0] = 1.0


def set_v_scales(c, scales):
    """V scales [pages, Hkv, 4] of a block-scaled cache; below 2^-100 they count as zero."""
    c.scale[:, :, 1] = scales
    counted = c.scale.numpy().copy()
    v = counted[:, :, 1]
    v[v < 2.0 ** -100] = 0.0
    c.vf = bc.values(c.v.view(torch.uint8).numpy(), counted, 1)


def check_scaled(c, got, log2):
    """check_shared of the output and the reference times 2^log2 (exact): small values count."""
    ref, mass = c.reference()
    f = 2.0 ** log2
    check_shared(got.double() * f, ref * f, mass * f, c.kv)


@pytest.mark.parametrize("B", [9, 20])
@pytest.mark.parametrize("log2", [100, -100])
def test_v_scales_at_both_ends_of_their_range(B, log2):
    """Scales of 2^100 and 2^-100, codes of 448 in half of the dims: over the 150 pages of one
    descriptor (or 75 of a half) their sums with weights of up to 2^8 pass 2^128.  The first
    page's scores stand 8 (log2) below the others: the softmax's reference is the first page's,
    or was when it was used."""
    lens = [64 * 150 + 1 + 5 * r for r in range(B)]
    c = Shared("block", lens, [0, B], [150], 8, 1, 1, seed=30 + B, poison=False)
    set_keys(c, [0.0] + [7.9 / 8 / 1.4426950408889634 * 128 ** 0.5] * 149, 7.5)
    step = float(c.k[int(c.table[0, 1]), 0, 0, 0].float())  # (as E4M3 holds it)
    assert 7.0 < 8 * step * c.sm * 1.4426950408889634 < 8.0
    c.v.view(torch.uint8)[..., ::2] = 0x7E  # 448
    set_v_scales(c, 2.0 ** log2)
    c.to_gpu()
    for ctas in (2, 0):
        got, _ = c.step(ctas=ctas)
        check_scaled(c, got, -log2)


def test_a_v_scale_below_its_range_counts_as_zero():
    """In the shared pages as in a request's own."""
    lens = [64 * 40 + 70 * r for r in range(12)]
    c = Shared("block", lens, [0, 12], [40], 8, 2, 1, seed=40, poison=False)
    set_v_scales(c, 2.0 ** -101)
    c.to_gpu()
    got, _ = c.step()
    assert not torch.count_nonzero(got)
    # where only some do, the others' values are as large as ever, the weights' sum too
    rng = np.random.default_rng(1)
    scales = torch.from_numpy(np.where(rng.random((c.k.shape[0], 2, 4)) < 0.5, 2.0 ** -101, 0.25))
    c.scale = c.scale.cpu()
    c.v = c.v.cpu()
    set_v_scales(c, scales.float())
    c.to_gpu()
    got, _ = c.step()
    c.check(got)


@pytest.mark.parametrize("heads", [(8, 1, 1), (16, 2, 1), (12, 2, 2), (64, 8, 1)])
def test_the_error_over_block_scales_is_that_of_the_unshared_step(heads):
    """In the Euclidean norm.  Both round their output to BF16 (2^-8 at most, 2^-8 / sqrt 3 of a
    value's step in the mean); the unshared step's weights are off by up to 2^-9 + 2^-11, the
    heads' by 2^-11 (f16), so the shared step's error is not larger but for chance: over at least
    20,000 outputs 1 / sqrt(2 n) = 0.5%; four times that is allowed."""
    hq, hkv, n = heads
    rng = np.random.default_rng(3)
    lens = [64 * 30 + n + int(t) for t in rng.integers(0, 300, 24)]
    c = Shared("block", lens, [0, 24], [30], hq, hkv, n, seed=41).to_gpu()
    ref, _ = c.reference()

    def error(got):
        return np.linalg.norm(got.double().cpu().numpy().reshape(ref.shape) - ref)

    assert ref.size >= 20000
    shared, unshared = error(c.step()[0]), error(Case.step(c, ws=Case.workspace(c))[0])
    assert shared <= 1.02 * unshared, (shared / np.linalg.norm(ref), unshared / np.linalg.norm(ref))


@pytest.mark.parametrize("heads", [(8, 1, 1), (16, 1, 1), (16, 2, 1), (24, 2, 1)])
@pytest.mark.parametrize("down", [False, True])
def test_v_scales_that_change_by_more_than_a_float_holds(heads, down):
    """Pages of V scale 2^-90 and pages of 2^90 behind one another (either way round), all
    scores alike: the first kind is in the sum of the weights, so the result is the second
    kind's mean times its share."""
    hq, hkv, n = heads
    lens = [64 * 44 + 3 * r for r in range(10)]
    c = Shared("block", lens, [0, 10], [40], hq, hkv, n, seed=42, poison=False)
    c.k = torch.zeros(c.k.shape).to(E4M3)
    c.kf = np.zeros(c.kf.shape)
    low = torch.zeros(c.k.shape[0], dtype=torch.bool)
    for row in c.table:  # of each request's entries the first 20, or those behind
        low[[int(p) for p in (row[20:] if down else row[:20]) if p >= 0]] = True
    set_v_scales(c, torch.where(low, 2.0 ** -90, 2.0 ** 90)[:, None, None])
    c.to_gpu()
    for ctas in (2, 0):
        got, _ = c.step(ctas=ctas)  # over shared pages
        check_scaled(c, got, -90)
        got, _ = Case.step(c, ws=Case.workspace(c, ctas))  # each request by itself
        ref, mass = c.reference()
        check_attention(got.double() * 2.0 ** -90, ref * 2.0 ** -90, mass * 2.0 ** -90, "block")


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("B", [9, 20])
def test_not_a_number_in_a_value_that_weighs_nothing(kv, B):
    """NaN in V of a shared page whose scores lie so far below the tails' that the heads'
    partials weigh 2^-200: times zero it is NaN still, in that dim of the rows that see it.
    The other dims are what they are."""
    lens = [64 * 3 + 1 + 11 * r for r in range(B)] + [150]
    c = Shared(kv, lens, [0, B], [3], 16, 2, 1, seed=50 + B, poison=False)
    set_keys(c, [0.0] * 3, 208.0)
    assert 8 * 208 * c.sm * 1.44 > 200
    c.to_gpu()
    clean, ws = c.step()
    c.check(clean)
    page = c.table[0, 2]
    if kv == "bf16":
        c.v[page, 5, 1, 7] = float("nan")
    else:
        c.v.view(torch.uint8)[page, 5, 1, 7] = 0x7F
    got, _ = c.step(ws=ws)
    hit = torch.zeros(got.shape, dtype=torch.bool)
    hit[:B, :, 8:, 7] = True
    assert torch.equal(got.isnan().cpu(), hit)
    assert torch.equal(got.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("where", ["tail", "shared"])
@pytest.mark.parametrize("entry", [-3, 10 ** 6])
def test_a_bad_entry_is_page_0_and_other_rows_keep_their_bits(kv, where, entry):
    """An entry out of range in request 7's own pages, or in the row that the group's shared
    pages are looked up in (request 0's): page 0 is read in its place."""
    lens = [64 * 3 + 40 * r for r in range(9)] + [64 * 3 - 1, 0, 250]
    c = Shared(kv, lens, [0, 11], [3], 16, 2, 1, seed=60, poison=False).to_gpu()
    clean, ws = c.step()
    r, t, rows = (7, 3, [7]) if where == "tail" else (0, 1, list(range(9)))
    good = c.bt[r, t].item()
    c.bt[r, t] = entry
    got, _ = c.step(ws=ws, flags=4)
    c.table[rows, t] = 0
    c.check(got)
    others = [b for b in range(len(lens)) if b not in rows]
    assert torch.equal(got[others], clean[others])
    c.bt[r, t] = good
    again, _ = c.step(ws=ws)
    assert torch.equal(again, clean)
