"""What the windowed and block-scaled calls promise about maps, bins and repeats."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from _blocks import Case
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
