"""Windowed prompt attention of rows that one token dominates."""

import numpy as np
import pytest
import torch

from _blocks import Case
from test_gpu_window import run_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(2, 1), (1, 1), (3, 1)])
@pytest.mark.parametrize("window,q_len,L", [(1500, 140, 1700), (100, 60, 500), (250, 300, 1000)])
def test_a_dominating_token_keeps_its_value(heads, window, q_len, L):
    """One token of weight 2^(7 + f) beside a sink of weight 1, the others 2^-28: the
    output is nearly that token's value, however many pages the row sees.

    f is where BF16 rounds worst (2^f = 1 + 0.98 * 2^-8 becomes 1).  With weights
    w~ = w (1 + d), |d| <= 2^-8, in the products and in their sum alike, the output
    is off by sum d_j p_j (v_j - out), to first order: 2^-8 sum p_j |v_j - out|,
    (1 + 2^-7) for the rest.  Scores are single products: exact but for the scale's
    and the exponential's fp32 roundings, 1e-5 of a weight.  Sums and products in
    fp32: 2^-15 of the values for 2^9 terms.  The output is rounded to BF16: 2^-8 of
    itself."""
    Hq, Hkv = heads
    c = Case("bf16", [L], Hq, Hkv, q_len, window, 1, seed=61, poison=False)
    f = float(np.log2(1 + 0.98 * 2.0 ** -8))
    c.sm = (7 + f) * np.log(2.0)  # times a product of 1 is 7 + f in log2
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k.zero_()
    c.k[..., 0] = -4.0
    # a token that every query sees, or one for each window's length of queries
    every = range(L - window, L - q_len + 1)
    doms = [every[len(every) // 2]] if every else list(range(L - q_len - window // 2, L, window))
    for t in [0] + doms:
        c.k[c.table[0, t // 64], t % 64, :, 0] = 0.0 if t == 0 else 1.0
    c.v[c.table[0, 0], 0] = 0.0
    c.qf, c.kf, c.vf = (x.double().numpy() for x in (c.q, c.k, c.v))
    out = run_prefill(c.to_gpu()).double().cpu().numpy().reshape(1, q_len, Hq, 128)
    from oracle import window as ow
    see = ow.visible(L, q_len, window, 1)
    K, V = (ow.gather(x, c.table[0], L) for x in (c.kf, c.vf))
    worst = 0.0
    for h in range(Hq):
        k, v = K[:, h // (Hq // Hkv)], V[:, h // (Hq // Hkv)]
        x = np.where(see, c.qf[0, :, h] @ k.T * c.sm, -np.inf)
        e = np.exp(x - x.max(-1, keepdims=True))
        p = e / e.sum(-1, keepdims=True)
        ref = p @ v
        spread = np.stack([p[i] @ np.abs(v - ref[i]) for i in range(q_len)])
        mass = p @ np.abs(v)
        tol = (2.0 ** -8 * (1 + 2.0 ** -7) + 2e-5) * spread + (1e-5 + 2.0 ** -15) * mass + \
            2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + 1e-30
        worst = max(worst, (np.abs(out[0, :, h] - ref) / tol).max())
    assert worst <= 1.0, f"off by {worst:.2f} of the tolerance"
