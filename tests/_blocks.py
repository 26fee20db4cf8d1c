"""Helpers of the block-scaled cache's and the windowed attention's tests:
inputs, calls through the C ABI and comparison with the fp64 oracles."""

from __future__ import annotations

import numpy as np
import torch

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as b
from oracle import block_cache as bc
from oracle import rope_norm as rn
from oracle import window as ow

E4M3 = torch.float8_e4m3fn
DTYPE = {"bf16": hd.HPC_KV_BF16, "e4m3": hd.HPC_KV_FP8_E4M3, "block": hd.HPC_KV_E4M3_BLOCK}


def page_table(lens, rng, spare=2):
    """A random page order: (table [B, max_pages], -1 past a request's pages; pages)."""
    per = [-(-max(L, 0) // 64) for L in lens]
    total = sum(per) + spare
    perm = rng.permutation(total)
    table = np.full((len(lens), max(per + [1])), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(per):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, total


def to_pow2(a: torch.Tensor) -> torch.Tensor:
    """pow2_scale of each element, by the exponent field (checked against the
    oracle's loop in the CPU tests)."""
    bits = a.float().contiguous().view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return (e.clamp_min(1) << 23).view(torch.float32)


class Case:
    """One batch with a paged cache on the device and its fp64 values on the host.

    spread: log2 range over which the blocks' sizes vary (the block scales with
    them).  poison: tokens no query sees, pages that hold none that one sees
    (their table entries too) and unused scales are NaN or out of range."""

    def __init__(self, kv, lens, Hq, Hkv, q_len, window, sinks, seed, spread=4.0, poison=True):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.lens, self.Hq, self.Hkv = kv, list(lens), Hq, Hkv
        self.q_len, self.window, self.sinks = q_len, window, sinks
        self.sm = 128 ** -0.5
        self.table, P = page_table(lens, rng)
        B = len(lens)
        x = torch.randn((2, P, 64, Hkv, 128), generator=gen, dtype=torch.float32)
        size = torch.exp2((torch.rand((2, P, 4, Hkv), generator=gen) - 0.5) * spread)
        size[0] = size[0].clamp(0.25, 2.0)  # keys: scores of a few units
        x *= size.repeat_interleave(16, 2)[..., None]
        self.ks = self.vs = 1.0
        self.scale = None
        if kv == "bf16":
            self.k, self.v = x[0].bfloat16(), x[1].bfloat16()
            self.kf, self.vf = self.k.double().numpy(), self.v.double().numpy()
        elif kv == "e4m3":
            self.ks, self.vs = (float(np.float32(float(x[i].abs().max()) / 448.0)) for i in (0, 1))
            self.k = (x[0] / self.ks).clamp(-448, 448).to(E4M3)
            self.v = (x[1] / self.vs).clamp(-448, 448).to(E4M3)
            self.kf = self.k.float().double().numpy() * self.ks
            self.vf = self.v.float().double().numpy() * self.vs
        else:
            s = to_pow2(x.view(2, P, 4, 16, Hkv, 128).abs().amax((3, 5)))  # [2, P, 4, Hkv]
            codes = (x / s.repeat_interleave(16, 2)[..., None]).to(E4M3)
            self.k, self.v = codes[0], codes[1]
            self.scale = s.permute(1, 3, 0, 2).contiguous()  # [P, Hkv, 2, 4]
            self.kf, self.vf = (bc.values(codes[i].view(torch.uint8).numpy(), self.scale.numpy(), i)
                                for i in (0, 1))
        q = torch.randn((B, q_len, Hq, 128), generator=gen, dtype=torch.float32)
        if kv == "bf16":
            self.q, self.qs = q.bfloat16(), None
            self.qf = self.q.double().numpy()
        else:
            self.qs = (q.abs().amax(-1) / 448.0).float()
            self.q = (q / self.qs[..., None]).clamp(-448, 448).to(E4M3)
            self.qf = self.q.float().double().numpy() * self.qs.double().numpy()[..., None]
        if poison:
            self._poison()

    def _poison(self):
        """NaN in every slot no query of its request sees (K, V and, for whole
        blocks, the scales); bad entries for pages without a seen token."""
        P = self.k.shape[0]
        seen = np.zeros((P, 64), dtype=bool)
        for r, L in enumerate(self.lens):
            if L <= 0:
                continue
            some = ow.visible(L, self.q_len, self.window, self.sinks).any(0)
            for t in range(self.table.shape[1]):
                part = some[64 * t:64 * t + 64]
                if self.table[r, t] < 0:
                    continue
                if part.any():
                    seen[self.table[r, t], :len(part)] = part
                elif self.window:  # an evicted page: any entry may stand there
                    self.table[r, t] = -7 if t % 2 else P + 1000
        for c in (self.k, self.v):
            if c.dtype is E4M3:
                c.view(torch.uint8)[torch.from_numpy(~seen)] = 0x7F
            else:
                c[torch.from_numpy(~seen)] = float("nan")
        if self.scale is not None:
            dead = ~seen.reshape(P, 4, 16).any(2)  # [P, 4]
            bad = torch.from_numpy(dead)[:, None, None, :].expand(self.scale.shape)
            self.scale[bad] = float("nan")

    def to_gpu(self):
        for name in ("k", "v", "q", "qs", "scale"):
            t = getattr(self, name)
            setattr(self, name, None if t is None else t.cuda())
        self.bt = torch.from_numpy(self.table).cuda()
        self.sl = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return self

    def workspace(self, ctas=0):
        return hd.Workspace(len(self.lens), self.Hq, self.Hkv, num_ctas=ctas,
                            kv_dtype=DTYPE[self.kv], q_len=self.q_len)

    def step(self, ctas=0, floor=2, fused=True, ws=None, stream=None):
        """hpc_decode_step_win; the output [B, q_len, Hq, 128] and the workspace."""
        ws = ws or self.workspace(ctas)
        shape = (len(self.lens), self.q_len, self.Hq, 128)
        out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        hd.hpc_decode_step_win(self.q, self.qs, self.k, self.v, self.ks, self.vs, self.scale,
                               self.bt, self.sl, self.Hq, self.Hkv, self.q_len, self.window,
                               self.sinks, self.sm, ws.num_ctas, floor, ws.tmap, ws.part_o,
                               ws.part_lse, out, unit_done=ws.unit_done if fused else None,
                               stream=stream)
        torch.cuda.synchronize()
        assert not fused or int(torch.count_nonzero(ws.unit_done)) == 0
        assert ws.tmap.to_host()["flags"] == 0
        return out, ws

    def reference(self):
        return ow.attention(self.qf, self.kf, self.vf, self.table, self.lens, self.window,
                            self.sinks, self.sm)

    def check(self, got):
        ref, mass = self.reference()
        check_attention(got, ref, mass, self.kv)


def check_attention(got, ref, mass, kv):
    """|got - ref| within the roundings of the kernels.

    The weights are rounded to the product's type: BF16 2^-8 of the value (and
    once more in the normaliser, which sums the rounded ones), 2 u sum w |v|.
    The 8-bit kernels form a weight in f16 (2^-11) and split it into three E5M2
    parts, each rounding what the last left by 2^-3 (two bits of fraction): 2^-9
    in all, and the normaliser is exact: (2^-9 + 2^-11) sum w |v| < 2^-8.6 sum w
    |v|, below 2 u with u = 2^-9.5.  The f16 weights of a cache without block
    scales go through the same kernels.  Weights below 2^-14 of the largest are
    off by up to 2^-25 of it instead, over at most 4096 tokens here 2^-13 of the
    largest value.  The output is rounded to BF16: 2^-8 |out|.  Scores are fp32 sums of
    128 products, |x| < 32 in these inputs: 128 * 2^-24 * 32 = 2.5e-4 of the
    weight, doubled for the two exponentials (running maximum and merge)."""
    u = 2.0 ** -8 if kv == "bf16" else 2.0 ** -9.5
    tol = (2 * u + 5e-4) * mass + 2.0 ** -8 * np.abs(ref) + 1e-30
    if kv != "bf16":
        tol = tol + 2.0 ** -13 * np.abs(mass).max(-1, keepdims=True)
    g = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(g).all(), "non-finite output"
    worst = (np.abs(g - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, f"off by {worst:.2f} of the tolerance"


# ------------------------------------------------------------------ prologue
class Prologue:
    """Inputs of hpc_rope_norm_block for given (request, position) tokens."""

    def __init__(self, tokens, Hq, Hkv, B, max_pages, seed, q8=True, layout=0, norm_first=True,
                 pad=0, table=None, extra_pages=1):
        gen = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        N = len(tokens)
        R = Hq + 2 * Hkv
        self.Hq, self.Hkv, self.N, self.q8 = Hq, Hkv, N, q8
        self.layout, self.norm_first = layout, norm_first
        mag = torch.exp2(torch.rand((N, R, 1), generator=gen) * 6 - 3)
        rows = (torch.randn((N, R, 128), generator=gen) * mag).bfloat16()
        full = torch.full((max(N, 1), R * 128 + pad), float("nan"), dtype=torch.bfloat16)
        full[:N, :R * 128] = rows.view(N, R * 128)
        self.qkv_host, self.full = rows, full
        self.wq = (1 + torch.randn(128, generator=gen) / 4).bfloat16()
        self.wk = (1 + torch.randn(128, generator=gen) / 4).bfloat16()
        self.req = np.array([r for r, _ in tokens], dtype=np.int32)
        self.pos = np.array([p for _, p in tokens], dtype=np.int32)
        P = B * max_pages + extra_pages
        if table is None:
            table = rng.permutation(P)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        self.table, self.P = table, P
        # what the cache held before: codes at power-of-two scales, as earlier
        # calls left them
        x = rng.standard_normal((2, P, 64, Hkv, 128)) * np.exp2(rng.uniform(-6, 6, (2, P, 1, Hkv, 1)))
        self.codes0, self.scale0 = [], np.zeros((P, Hkv, 2, 4), dtype=np.float32)
        for i in range(2):
            t = torch.from_numpy(x[i]).float().view(P, 4, 16, Hkv, 128)
            s = to_pow2(t.abs().amax((2, 4)))
            c = (t / s[:, :, None, :, None]).view(P, 64, Hkv, 128).to(E4M3)
            self.codes0.append(c.view(torch.uint8).numpy().copy())
            self.scale0[:, :, i] = s.permute(0, 2, 1).numpy()

    def run(self, freq=None, **kw):
        N, Hq = self.N, self.Hq
        self.k, self.v = (torch.from_numpy(c.copy()).cuda().view(E4M3) for c in self.codes0)
        self.scale = torch.from_numpy(self.scale0.copy()).cuda()
        self.q = torch.full((max(N, 1), Hq, 128), float("nan"), dtype=torch.float32).to(
            E4M3 if self.q8 else torch.bfloat16).cuda()
        self.qs = torch.full((max(N, 1), Hq), float("nan")).cuda() if self.q8 else None
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        hd.hpc_rope_norm_block(
            self.full.cuda(), self.wq.cuda(), self.wk.cuda(), torch.from_numpy(self.pos).cuda(),
            torch.from_numpy(self.req).cuda(), Hq, self.Hkv, torch.from_numpy(self.table).cuda(),
            self.k, self.v, self.scale, self.q, self.qs, self.flags, rope_layout=self.layout,
            norm_first=self.norm_first, freq=freq, **kw)
        torch.cuda.synchronize()
        return self

    def exact_rows(self):
        """fp64 (q [N, Hq, 128], k [N, Hkv, 128], v) of the prologue."""
        x = self.qkv_host.double().numpy()
        Hq, Hkv = self.Hq, self.Hkv
        q, k = np.zeros((self.N, Hq, 128)), np.zeros((self.N, Hkv, 128))
        for t in range(self.N):
            a = (int(self.pos[t]), float(np.float32(1e-6)), 1e6, self.layout, self.norm_first)
            q[t] = rn.norm_and_rope(x[t, :Hq], self.wq.double().numpy(), *a)
            k[t] = rn.norm_and_rope(x[t, Hq:Hq + Hkv], self.wk.double().numpy(), *a)
        return q, k, x[:, Hq + Hkv:]

    def oracle_write(self, k, v):
        """The oracle's (codes, scales) pair for rows k, v; runs; flags."""
        out = []
        for i, rows in enumerate((k, v)):
            out.append(bc.write(rows, self.pos, self.req, self.table, self.codes0[i],
                                self.scale0[:, :, i]))
        return out


PAGE_BYTES = b.PAGE_SIZE * b.HEAD_DIM
