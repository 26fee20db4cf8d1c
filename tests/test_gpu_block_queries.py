"""FP8 query rows of the prologues (hpc_rope_norm_block, hpc_rope_norm) at the ends of
fp32's range."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from _blocks import Prologue

pytestmark = pytest.mark.gpu


def run(pro, block):
    """The prologue of either cache (one scale per cache: 1) on pro's inputs."""
    if block:
        return pro.run()
    gpu = lambda x: (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()  # noqa: E731
    k, v = (torch.from_numpy(c.copy()).cuda().view(torch.float8_e4m3fn) for c in pro.codes0)
    pro.q = torch.full((pro.N, pro.Hq, 128), float("nan")).to(torch.float8_e4m3fn).cuda()
    pro.qs = torch.full((pro.N, pro.Hq), float("nan")).cuda()
    hd.hpc_rope_norm(gpu(pro.full), gpu(pro.wq), gpu(pro.wk), gpu(pro.pos), gpu(pro.req), pro.Hq,
                     pro.Hkv, gpu(pro.table), k, v, 1.0, 1.0, pro.q, pro.qs)
    torch.cuda.synchronize()
    return pro


@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("log2_size", [-123, -121, -119, -117, -101, -100, -99, 99, 101, 119, 120])
def test_query_rows_of_any_size(log2_size, block):
    """Rows whose largest value is about 2^log2_size, with exact zeros: 448 / max
    passes fp32's range below 2^-119.

    Codes are E4M3 of y * 448 / max: half a step is 2^-4 of the value, 2^-10 of
    the scale for subnormal codes.  fp32 before that: the norm and the rotation
    4e-6 of the row's largest value (128 squares, a root, three products, two
    terms of the rotation), the quotient and its product 4 * 2^-24 of the value.
    The scale max * (1 / 448) rounds twice, 2^-23 of itself, or to a multiple of
    2^-149, which a code multiplies by up to 448."""
    pro = Prologue([(0, p) for p in range(5)], 4, 1, 1, 1, seed=abs(log2_size))
    rows = pro.qkv_host
    rows[:, :4, 3::7] = 0.0
    rows[:, :4, 64 + 3::7] = 0.0
    # the norm makes rows of mean square 1; the weights size them
    pro.wq = (pro.wq.float() * 2.0 ** log2_size).bfloat16()
    pro.full = rows.view(5, -1)
    run(pro, block)
    q, _, _ = pro.exact_rows()
    big = np.abs(q).max(-1, keepdims=True)
    got = pro.q[:5].float().cpu().double().numpy()
    s = pro.qs[:5].cpu().double().numpy()[..., None]
    assert np.isfinite(got).all() and np.isfinite(s).all()
    want = big / 448
    if not block:  # the least maximum before the norm's factor, documented
        x = pro.qkv_host[:, :4].double().numpy()
        inv = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(1e-6)))
        want = np.maximum(big, 1.3166e-36 * inv) / 448
    assert (np.abs(s - want) <= (2 * 4e-6 + 2.0 ** -23) * want + 2.0 ** -149).all()
    tol = (2.0 ** -4 + 2.0 ** -22) * np.abs(q) + 2.0 ** -10 * s + 2 * 4e-6 * big + 448 * 2.0 ** -149
    assert (np.abs(got * s - q) <= tol).all()
    assert (got[q == 0.0] == 0.0).all()


@pytest.mark.parametrize("block", [True, False])
def test_subnormal_inputs_beside_zeros(block):
    """BF16-subnormal values next to exact zeros (eps, not the row, sets the norm)."""
    pro = Prologue([(0, 0)], 2, 1, 1, 1, seed=5)
    rows = torch.zeros_like(pro.qkv_host)
    rows[0, 0, 7], rows[0, 1, 100] = 2.0 ** -130, -(2.0 ** -133)
    pro.full = rows.view(1, -1)
    run(pro, block)
    got, s = pro.q.float().cpu().double(), pro.qs.cpu().double()
    want = torch.zeros_like(got)
    for h, d in ((0, 7), (1, 100)):
        want[0, h, d] = float(rows[0, h, d].double() * pro.wq[d].double()) / np.sqrt(
            float(np.float32(1e-6)))
    # position 0: nothing is turned; one value a row, whose code is +-448.  Its
    # product with the norm's weight is rounded to a multiple of 2^-149 and then
    # multiplied by 1000, its scale to one and by 448.
    assert torch.isfinite(got).all()
    code = torch.zeros_like(want)
    if block:
        assert torch.equal(got != 0, want != 0) and (got.abs().amax(-1) == 448).all()
    else:  # codes by the least maximum's scale: half a step of theirs
        assert torch.allclose(s, torch.full_like(s, 1.3166e-36 / np.sqrt(1e-6) / 448), rtol=1e-5)
        code = 2.0 ** -4 * want.abs() + 2.0 ** -10 * s[..., None]
    tol = code + 4e-6 * want.abs() + (500 + 448) * 2.0 ** -149
    assert ((got * s[..., None] - want).abs() <= tol).all()
