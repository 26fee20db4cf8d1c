"""Pins of the windowed-attention and block-cache oracles (CPU only)."""

import numpy as np
import pytest
import torch

import oracle
from _blocks import to_pow2
from oracle import block_cache as bc
from oracle import rope_norm as rn
from oracle import window as ow


def naive_visible(L, n, W, S):
    out = np.zeros((n, L), dtype=bool)
    for i in range(n):
        p = L - n + i
        for j in range(L):
            out[i, j] = j <= p and (W == 0 or p - j < W or j < S)
    return out


@pytest.mark.parametrize("L,n,W,S", [(1, 1, 1, 0), (5, 7, 2, 1), (40, 3, 8, 4), (40, 3, 0, 0),
                                     (70, 70, 1, 0), (70, 5, 100, 3), (9, 2, 3, 50)])
def test_visible_is_the_definition(L, n, W, S):
    assert np.array_equal(ow.visible(L, n, W, S), naive_visible(L, n, W, S))


def test_attention_without_a_window_is_the_other_oracle():
    rng = np.random.default_rng(3)
    lens = [1, 64, 65, 130]
    q = torch.from_numpy(rng.standard_normal((4, 2, 4, 128))).bfloat16()
    k = torch.from_numpy(rng.standard_normal((9, 64, 2, 128))).bfloat16()
    v = torch.from_numpy(rng.standard_normal((9, 64, 2, 128))).bfloat16()
    table = np.array([[3, 0, 0], [1, 0, 0], [8, 2, 0], [5, 7, 4]], dtype=np.int32)
    ref = oracle.attention_mq(q, k, v, table, lens, 2, num_q_heads=4, num_kv_heads=2,
                              sm_scale=0.1)
    got, _ = ow.attention(q.double().numpy(), k.double().numpy(), v.double().numpy(), table, lens,
                          0, 0, 0.1)
    assert np.abs(got - ref).max() < 1e-12


def test_a_window_of_one_is_the_value_row():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal(s) for s in ((1, 3, 2, 128), (2, 64, 1, 128), (2, 64, 1, 128)))
    got, _ = ow.attention(q, k, v, np.array([[1, 0]]), [70], 1, 0, 0.1)
    for i, t in enumerate((67, 68, 69)):
        row = v[0, t - 64, 0]
        assert np.allclose(got[0, i], row)


@pytest.mark.parametrize("W,S,n", [(1, 0, 1), (64, 0, 1), (65, 1, 2), (128, 64, 1), (100, 70, 4),
                                   (1000, 3, 1)])
def test_planned_lengths_keep_every_visible_tile(W, S, n):
    for L in list(range(0, 400, 7)) + [640, 641, 4096]:
        got = ow.planned_lengths([L], 64, n, W, S)[0]
        see = ow.visible(L, n, W, S).any(0) if L else np.zeros(0, bool)
        tiles = sum(see[64 * t:64 * t + 64].any() for t in range(-(-L // 64)))
        # (a tile between may be kept when L < q_len: nothing is left out then)
        assert -(-got // 64) >= tiles
        if L >= n:
            assert -(-got // 64) == max(tiles, 0), (L, got, tiles)
        assert got % 64 == L % 64


def test_pow2_scale_against_the_exponent_field():
    a = torch.cat([torch.tensor([0.0, 448.0, 448.5, 447.9, 1.75, 1.7500001, 3.5, 1e-40, 1e-38,
                                 2.0 ** -126 * 448, 3.3e38]),
                   torch.exp2(torch.linspace(-120, 120, 400))])
    want = torch.tensor([bc.pow2_scale(float(x)) for x in a], dtype=torch.float64)
    assert torch.equal(to_pow2(a).double(), want)


def test_write_fresh_append_and_growth():
    rng = np.random.default_rng(6)
    table = np.array([[2, 0], [1, 3]], dtype=np.int32)
    codes = np.zeros((4, 64, 1, 128), dtype=np.uint8)
    scales = np.full((4, 1, 4), np.nan)
    first = rng.standard_normal((5, 1, 128))
    c1, s1, runs, flags = bc.write(first, range(5), [0] * 5, table, codes, scales)
    assert flags == 0 and runs == [(2, 0, [0, 1, 2, 3, 4])]
    assert s1[2, 0, 0] == bc.pow2_scale(np.abs(first).max())
    assert np.abs(rn.e4m3_decode(c1[2, :5, 0]) * s1[2, 0, 0] - first[:, 0]).max() <= \
        2.0 ** -4 * np.abs(first).max()
    # a larger token grows the scale; the earlier codes follow
    big = 64 * rng.standard_normal((1, 1, 128))
    c2, s2, _, _ = bc.write(big, [5], [0], table, c1, s1)
    assert s2[2, 0, 0] > s1[2, 0, 0]
    old, new = (rn.e4m3_decode(c[2, :5, 0]) * s[2, 0, 0] for c, s in ((c1, s1), (c2, s2)))
    assert np.abs(old - new).max() <= s2[2, 0, 0] * 2.0 ** -10  # half a subnormal step
    # a smaller one leaves scale and codes alone
    c3, s3, _, _ = bc.write(big / 1e3, [6], [0], table, c2, s2)
    assert s3[2, 0, 0] == s2[2, 0, 0] and np.array_equal(c3[2, :6], c2[2, :6])
    # the block's first position starts it afresh
    c4, s4, _, _ = bc.write(first[:1] / 1e3, [0], [0], table, c3, s3)
    assert s4[2, 0, 0] == bc.pow2_scale(np.abs(first[0]).max() / 1e3)


def test_write_flags_and_runs():
    table = np.array([[0, 9], [1, -1]], dtype=np.int32)
    codes, scales = np.zeros((2, 64, 1, 128), np.uint8), np.ones((2, 1, 4))
    rows = np.ones((6, 1, 128))
    _, _, runs, flags = bc.write(rows, [15, 16, 64, -1, 3, 200], [0, 0, 0, 0, 1, 1], table, codes,
                                 scales)
    assert flags == 5 and [r[2] for r in runs] == [[0], [1], [4]]
    _, _, runs, flags = bc.write(np.ones((17, 1, 128)), list(range(16)) + [3], [0] * 17, table,
                                 codes, scales)
    assert flags == 1 and len(runs) == 1 and len(runs[0][2]) == 16


def test_infinities_and_nan_in_a_run():
    rows = np.ones((1, 1, 128))
    rows[0, 0, 3], rows[0, 0, 4], rows[0, 0, 5] = np.inf, np.nan, -np.inf
    c, s, _, _ = bc.write(rows, [0], [0], np.array([[0]]), np.zeros((1, 64, 1, 128), np.uint8),
                          np.ones((1, 1, 4)))
    got = rn.e4m3_decode(c[0, 0, 0])
    assert s[0, 0, 0] == bc.pow2_scale(1.0)
    assert got[3] == 448 and np.isnan(got[4]) and got[5] == -448 and got[0] * s[0, 0, 0] == 1.0
