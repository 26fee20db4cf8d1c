"""The block-scaled decode's softmax sum at its ends."""

import numpy as np
import pytest
import torch

from _blocks import Case
from oracle import block_cache as bc

pytestmark = pytest.mark.gpu


def test_tiny_v_scales_over_tens_of_millions_of_tokens():
    """One request whose block table names the same few pages over and over, on one
    CTA.  V's scales are 2^-100, which the softmax's reference takes as 2^-88: a weight
    of 2^11.2 above the first tokens' stands for 2^(88 + 3 + 11.2) in the sum, and
    2^26 of them for 2^128.2 (2^127.2 in each half).

    All values are the same, so the output is that value whatever the weights:
    rounded by 2^-8 (BF16), by 2^-9 for the weights' three parts, and by the fp32
    accumulator, whose 2^21 additions may each cut off 2^-23 of what it holds (half of
    the final sum on average): 2^-3."""
    c = Case("block", [640], 1, 1, 1, 0, 0, seed=44, poison=False)
    c.k.view(torch.uint8).zero_()
    rows = c.table[0]
    c.k.view(torch.uint8)[torch.from_numpy(rows[4:]), :, :, 0] = 0x38  # 1.0 from token 256 on
    c.v.view(torch.uint8).fill_(0x38)
    c.q.view(torch.uint8).zero_()
    c.q.view(torch.uint8)[..., 0] = 0x38
    c.qs.fill_(11.2 * np.log(2.0) / c.sm)
    c.scale[:, :, 0], c.scale[:, :, 1] = 1.0, 2.0 ** -100
    pages = 1 << 20
    more = torch.from_numpy(np.resize(rows[4:], pages - 4))
    c.table = torch.cat([torch.from_numpy(rows[:4].copy()), more])[None].int().numpy()
    c.lens = [64 * pages]
    c.to_gpu()
    got, ws = c.step(ctas=1)
    value = got.double() * 2.0 ** 100
    assert ((value - 1).abs() <= 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -3).all()
    c.step(ctas=1, fused=False, ws=ws)
    want = np.log(2.0) * (26 + 11.2)
    # a sum of 2^26 terms, each thread's and then theirs: 2^18 additions of 2^-24
    assert abs(float(ws.part_lse[0, 0]) - want) <= 2.0 ** -6


def check_over(got, ref, mass, tokens):
    """check_attention's bound for 8-bit caches with its absolute part for `tokens`
    weights (each below 2^-14 of the largest off by up to 2^-25 of it)."""
    extra = tokens * 2.0 ** -25 * np.abs(mass).max(-1, keepdims=True)
    tol = (2.0 ** -9 + 2.0 ** -11 + 5e-4) * mass + 2.0 ** -8 * np.abs(ref) + extra + 1e-30
    g = got.double().cpu().numpy().reshape(ref.shape)
    worst = (np.abs(g - ref) / tol).max()
    assert worst <= 1.0, f"off by {worst:.2f} of the tolerance"


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -90])
def test_tiny_v_scales_over_more_tokens(scale):
    """60,000 tokens whose weights stand 2^11.2 above the first ones': taken at its own
    size, a scale of 2^-100 would make each half's sum 30,000 * 2^(100 + 3 + 11.2),
    past 2^128."""
    n = 60000
    c = Case("block", [n], 8, 1, 1, 0, 0, seed=45, poison=False)
    c.k.view(torch.uint8).zero_()
    c.k.view(torch.uint8)[torch.from_numpy(c.table[0][4:]), :, :, 0] = 0x38
    c.q.view(torch.uint8).zero_()
    c.q.view(torch.uint8)[..., 0] = 0x38
    c.qs.fill_(11.2 * np.log(2.0) / c.sm)
    s = c.scale.numpy()
    s[:, :, 0], s[:, :, 1] = 1.0, scale
    c.qf = c.q.float().double().numpy() * c.qs.double().numpy()[..., None]
    c.kf, c.vf = (bc.values(x.view(torch.uint8).numpy(), s, i) for i, x in enumerate((c.k, c.v)))
    got, _ = c.to_gpu().step(ctas=1)
    ref, mass = c.reference()
    check_over(got.double() / scale, ref / scale, mass / scale, n)


@pytest.mark.parametrize("kv", ["e4m3", "block"])
def test_long_windows_within_their_own_bound(kv):
    """Windows of 6000 and sinks: the small weights' part of the bound is for all of
    the tokens that a query sees."""
    c = Case(kv, [20000, 70, 9000], 8, 1, 1, 6000, 130, seed=63).to_gpu()
    ref, mass = c.reference()
    for ctas in (0, 400, 1):
        got, _ = c.step(ctas=ctas)
        check_over(got, ref, mass, 6130)


def test_a_window_beyond_every_length_and_the_plain_step_of_e4m3():
    """The windowed kernel's weights are three E5M2 parts (2^-9 and, in f16, 2^-11) and
    its sum exact; the plain one's are f16 in both (2^-11 twice)."""
    c = Case("e4m3", [1, 64, 700, 3000, 0], 8, 1, 1, 4000, 0, seed=8, poison=False).to_gpu()
    got, _ = c.step()
    c.window = 0
    plain, _ = c.step()
    ref, mass = c.reference()
    weights = 2.0 ** -9 + 2.0 ** -11 + 2 * 2.0 ** -11 + 1e-3 + 3000 * 2.0 ** -25
    far = (got.double() - plain.double()).abs().cpu().numpy().reshape(mass.shape)
    big = np.abs(mass).max(-1, keepdims=True)
    assert (far <= weights * big + 2 * 2.0 ** -8 * (np.abs(ref) + weights * big) + 1e-30).all()
