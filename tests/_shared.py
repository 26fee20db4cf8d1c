"""Helpers of the shared-prefix decode's tests."""

from __future__ import annotations

import numpy as np
import torch

import load_balanced_paged_assign_gb300 as hd
from _blocks import DTYPE, Case


class Shared(Case):
    """A batch whose groups share pages: group g is requests starts[g] .. starts[g + 1] - 1,
    the first pages[g] entries of those that reach past them name the same pages."""

    def __init__(self, kv, lens, starts, pages, Hq, Hkv, q_len, seed, spread=4.0, poison=True):
        super().__init__(kv, lens, Hq, Hkv, q_len, 0, 0, seed, spread=spread, poison=poison)
        self.starts, self.pages = list(starts), list(pages)
        self.lead = {}
        for g, n in enumerate(self.pages):
            who = [r for r in range(starts[g], starts[g + 1]) if self.sees(r, n)]
            for r in who:
                self.table[r, :n] = self.table[who[0], :n]
                if len(who) > 1:
                    self.lead[r] = (g, n)

    def sees(self, r, n):
        """All queries of request r see n pages."""
        return n > 0 and self.lens[r] - self.q_len + 1 >= 64 * n

    def workspace(self, ctas=0):
        return hd.SharedWorkspace(len(self.lens), self.Hq, self.Hkv, len(self.pages),
                                  num_ctas=ctas, kv_dtype=DTYPE[self.kv], q_len=self.q_len)

    def groups(self):
        return (torch.tensor(self.starts, dtype=torch.int32).cuda(),
                torch.tensor(self.pages, dtype=torch.int32).cuda())

    def out(self):
        return torch.full((len(self.lens), self.q_len, self.Hq, 128), float("nan"),
                          dtype=torch.bfloat16, device="cuda")

    def step(self, ctas=0, floor=2, ws=None, stream=None, flags=0):
        ws = ws or self.workspace(ctas)
        ws.head_o.fill_(float("nan"))  # what is not written is not read
        ws.part_o.fill_(float("nan"))
        out, (starts, pages) = self.out(), self.groups()
        torch.cuda.synchronize()
        hd.hpc_decode_step_shared(self.q, self.qs, self.k, self.v, self.ks, self.vs, self.scale,
                                  self.bt, self.sl, starts, pages, self.Hq, self.Hkv, self.q_len,
                                  self.sm, floor, ws, out, stream=stream)
        torch.cuda.synchronize()
        assert ws.flags == flags
        return out, ws

    def check(self, got):
        ref, mass = self.reference()
        check_shared(got, ref, mass, self.kv)

    def check_plan(self, ws):
        """Every tile of every request is some descriptor's, once, and no CTA's share is
        over its budget."""
        B, C, Hkv, G = len(self.lens), ws.num_ctas, self.Hkv, self.Hq // self.Hkv
        tpb = 128 // G
        h = ws.head.tolist()
        ctas, num, budget = h[:3]
        with_ = min(ws.num_groups if not hasattr(self, "n") else self.n, B // 2)
        units = Hkv * (B * self.q_len // (2 * tpb) + with_) if with_ else 0
        at = 8
        req = [h[at + 4 * r:at + 4 * r + 4] for r in range(B)]
        at += 4 * B
        bins = h[at:at + C + 1]
        at += (C + 1 + 3) // 4 * 4
        unit = [h[at + 2 * u:at + 2 * u + 2] for u in range(h[4])]
        at += (2 * units + 3) // 4 * 4
        desc = [h[at + 8 * d:at + 8 * d + 8] for d in range(num)]
        assert bins[0] == 0 and bins[ctas:] == [num] * (C + 1 - ctas)
        assert all(a < b for a, b in zip(bins[:ctas], bins[1:ctas + 1]))
        for c in range(ctas):
            # (8 a page of two row tiles, 5 one of a tile alone; the last may reach over)
            cost = [(d[5] - d[4], 8 if d[6] else 5) for d in desc[bins[c]:bins[c + 1]]]
            assert sum(n * w for n, w in cost) < budget + cost[-1][1]
        seen = [0] * num
        tail = ws.tmap.to_host()
        two = 2 if self.kv != "bf16" and Hkv % 2 == 0 else 1
        for r, L in enumerate(self.lens):
            skip = self.lead[r][1] if r in self.lead else 0
            assert req[r][0] == skip
            for hp in range(Hkv // two):
                u = hp * B + r
                tiles = []
                for d in range(tail["chunk_off"][u], tail["chunk_off"][u] + tail["chunk_count"][u]):
                    assert tail["desc"][d][:2] == (hp, r)
                    tiles += range(*tail["desc"][d][2:])
                assert tiles == list(range(skip, -(-L // 64)))
            if not skip:
                continue
            for i in range(self.q_len):
                for k in range(Hkv):
                    tok = r * self.q_len + i - req[r][2]
                    t = tok // tpb
                    off, cnt = unit[req[r][1] + k * ((req[r][3] + 1) // 2) + t // 2]
                    tiles = []
                    for d in range(off, off + cnt):
                        x = desc[d]
                        assert x[0] == k and x[1] == req[r][2] + 2 * (t // 2) * tpb
                        assert x[1] + (t % 2) * tpb <= r * self.q_len + i < x[2]
                        assert t % 2 <= x[6] and x[7] == 0
                        assert self.lead[x[3]][0] == self.lead[r][0]
                        tiles += range(x[4], x[5])
                        seen[d] = 1
                    assert tiles == list(range(skip))
        assert all(seen)
        for c in range(C):
            b = tail["bin_ptr"][c:c + 2]
            assert b[0] <= b[1] and (c >= ctas or b == [0, 0])
            assert sum(x[3] - x[2] for x in tail["desc"][b[0]:b[1]]) <= tail["budget"]
        assert tail["bin_ptr"][C] == tail["num_desc"]


def check_shared(got, ref, mass, kv):
    """|got - ref| within the roundings of the kernels, u sum w |v| for the weights:
    BF16 pages: rounded to BF16, 2^-8, and again in the normaliser: 2 * 2^-8.
    E4M3: f16 and in the normaliser, 2 * 2^-11, in the head; three E5M2 parts of an f16
    weight, 2^-9 + 2^-11, in the tail: 2^-8.6 at most.
    Block scales: rounded to BF16 with the block's scale, the normaliser exact: 2^-8 in
    the head, 2^-8.6 in the tail.
    The head's f16 weights below 2^-14 of the type are off by 2^-25 at most, times 2^-6
    of their scale; the tail's as in check_attention: over at most 4096 tokens 2^-13 of
    the largest value.  Scores are fp32 sums of 128 products, |x| < 32: 128 * 2^-24 * 32 =
    2.5e-4 of the weight, doubled for the exponentials (running maximum, join).  The
    output is rounded to BF16: 2^-8 |out|."""
    u = {"bf16": 2.0 ** -7, "e4m3": 2.0 ** -8.6, "block": 2.0 ** -8}[kv]
    tol = (u + 5e-4) * mass + 2.0 ** -8 * np.abs(ref) + 1e-30
    if kv != "bf16":
        tol = tol + 2.0 ** -13 * np.abs(mass).max(-1, keepdims=True)
    g = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(g).all(), "non-finite output"
    worst = (np.abs(g - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, f"off by {worst:.2f} of the tolerance"
