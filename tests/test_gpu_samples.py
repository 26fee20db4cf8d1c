"""The page pool and the shared-prefix decode as a runtime uses them: a prompt is written,
samples are forked from it, grow, decode over the shared pages, end, and the cache is
brought together."""

import numpy as np
import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from _shared import check_shared
from load_balanced_paged_assign_gb300 import binding as E
from oracle import window as ow

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def ints(x):
    return torch.tensor(x, **I32)


class Server:
    """Rows of a table on a pool, one layer's cache, and every row's K and V on the host."""

    def __init__(self, rows, max_pages, pages, Hq, Hkv, kv):
        self.Hq, self.Hkv, self.kv = Hq, Hkv, kv
        self.pool = hd.PagePool(pages)
        self.table = torch.full((rows, max_pages), -1, **I32)
        self.copies = torch.zeros((pages + rows + 1, 2), **I32)
        dtype = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
        shape = (pages, 64, Hkv, 128)
        self.k, self.v = (torch.zeros(shape, device="cuda").to(dtype) for _ in range(2))
        self.scale = torch.zeros((pages, Hkv, 2, 4), device="cuda") if kv == "block" else None
        self.len = [0] * rows
        self.gen = torch.Generator(device="cuda").manual_seed(3)
        self.w = torch.ones(128, device="cuda").bfloat16()

    def append(self, rows, counts):
        """New tokens through the prologue; returns the queries of the last token of each row."""
        want = [self.len[r] + n for r, n in zip(rows, counts)]
        hd.hpc_kv_extend(self.pool, self.table, ints(rows), ints(want))
        req = [r for r, n in zip(rows, counts) for _ in range(n)]
        pos = [self.len[r] + i for r, n in zip(rows, counts) for i in range(n)]
        N = len(req)
        qkv = torch.randn((N, (self.Hq + 2 * self.Hkv) * 128), generator=self.gen,
                          device="cuda").bfloat16()
        q8 = self.kv != "bf16"
        q = torch.zeros((N, self.Hq, 128), device="cuda").to(self.k.dtype)
        qs = torch.zeros((N, self.Hq), device="cuda") if q8 else None
        if self.kv == "block":
            hd.hpc_rope_norm_block(qkv, self.w, self.w, ints(pos), ints(req), self.Hq, self.Hkv,
                                   self.table, self.k, self.v, self.scale, q, qs)
        else:
            hd.hpc_rope_norm(qkv, self.w, self.w, ints(pos), ints(req), self.Hq, self.Hkv,
                             self.table, self.k, self.v, 0.02, 0.02, q, qs)
        for r, L in zip(rows, want):
            self.len[r] = L
        last = [i for i in range(N) if i + 1 == N or req[i + 1] != req[i]]
        return q[last].contiguous(), None if qs is None else qs[last].contiguous()

    def values(self):
        """fp64 (K, V) pages on the host."""
        if self.kv == "bf16":
            return self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        if self.kv == "e4m3":
            return (self.k.float().double().cpu().numpy() * np.float32(0.02).astype(float),
                    self.v.float().double().cpu().numpy() * np.float32(0.02).astype(float))
        from oracle import block_cache as bc
        s = self.scale.cpu().numpy()
        return tuple(bc.values(c.view(torch.uint8).cpu().numpy(), s, i)
                     for i, c in enumerate((self.k, self.v)))

    def decode(self, rows, q, qs, starts, pages, ws):
        out = torch.full((len(rows), 1, self.Hq, 128), float("nan"), dtype=torch.bfloat16,
                         device="cuda")
        table, lens = self.table[rows].contiguous(), ints([self.len[r] for r in rows])
        scale = 0.02 if self.kv == "e4m3" else 1.0
        hd.hpc_decode_step_shared(q, qs, self.k, self.v, scale, scale, self.scale, table, lens,
                                  ints(starts), ints(pages), self.Hq, self.Hkv, 1, 128 ** -0.5, 2,
                                  ws, out)
        torch.cuda.synchronize()
        assert ws.flags == 0 and self.pool.flags == 0
        qf = q.float().double().cpu().numpy()
        if qs is not None:
            qf = qf * qs.double().cpu().numpy()[..., None]
        K, V = self.values()
        ref, mass = ow.attention(qf[:, None], K, V, table.cpu().numpy(), lens.tolist(), 0, 0,
                                 128 ** -0.5)
        check_shared(out, ref, mass, self.kv)
        return out


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "block"])
def test_samples_of_two_prompts(kv):
    s = Server(24, 12, 200, 16, 2, kv)
    s.append([0, 1], [300, 130])
    # nine samples of the first prompt and six of the second, which end inside a page
    src, dst = [0] * 9 + [1] * 6, list(range(2, 17))
    lens = [s.len[a] for a in src]
    hd.hpc_kv_fork(s.pool, s.table, ints(src), ints(dst), ints(lens), s.copies)
    hd.hpc_kv_copy_pages(s.copies, s.k, s.v, s.scale)
    for b, L in zip(dst, lens):
        s.len[b] = L
    assert int(s.pool.refs[s.table[0, 0].long()]) == 10
    ws = hd.SharedWorkspace(15, 16, 2, 2, kv_dtype={"bf16": 0, "e4m3": 1, "block": 2}[kv])
    rng = np.random.default_rng(0)
    for step in range(3):  # they grow at their own pace, into pages of their own
        q, qs = s.append(dst, [int(n) for n in rng.integers(1, 70, len(dst))])
        s.decode(dst, q, qs, [0, 9, 15], [300 // 64, 130 // 64], ws)
    assert ws.head_ctas() > 0
    # some end; the others go on from a cache without holes
    hd.hpc_kv_free(s.pool, s.table, ints([1, 3, 4, 8, 12, 13]))
    for r in (1, 3, 4, 8, 12, 13):
        s.len[r] = 0
    left = [r for r in dst if s.len[r] > 0]
    before = [len(set(s.table[left].flatten().tolist()) - {-1}), s.pool.free_pages]
    hd.hpc_kv_compact(s.pool, s.table, s.copies)
    hd.hpc_kv_copy_pages(s.copies, s.k, s.v, s.scale)
    assert s.pool.free_pages == before[1]
    assert int(s.table.max()) < 200 - before[1]
    q, qs = s.append(left, [1] * len(left))
    s.decode(left, q, qs, [0, sum(r < 11 for r in left), len(left)], [4, 2], ws)
    hd.hpc_kv_free(s.pool, s.table)
    assert s.pool.free_pages == 200 and s.pool.flags == 0
    assert E.HPC_FLAG_NO_PAGES == 16
