"""Decode over shared prefixes and the pages of a cache, as measured.

Every case is one pass through what a serving runtime does with requests that
begin alike: a decode step whose requests share the pages of a prompt (in
groups, over BF16, E4M3 or block-scaled pages), children that are forked from
the pages of their parents (those that end are freed first, and the page that a
child will write to is copied), requests that leave and make room for others,
and the moves that bring a fragmented cache's live pages together.

`run` computes the operator in plain torch operations (32 bits, rounded once at
the end) where `own` is false, and calls the framework where it is true.  Caches
are [pages, 64, Hkv, 128]; block scales [pages, Hkv, 2, 4] hold K's four scales
of a page and then V's.  A pool of pages is `refs` (the rows that hold a page),
`free` (a stack of the pages that none holds, the next one to be handed out at
free[state[0] - 1]) and `state` ({free pages, flags, 0, 0}).
"""

import math
import random

import torch

own = False

D = 128
PAGE = 64
BLOCK = 16
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few users behind one system prompt, the latency of a small step
        dict(name="shared_small", op="attn", kv="bf16", B=4, Hq=8, Hkv=1, q_len=1, groups=1,
             loose=0, pre_lo=15, pre_hi=15, tail_lo=20, tail_hi=200, lens=1),
        # a full batch behind one long system prompt, all heads on one GPU
        dict(name="shared_prompt_8k", op="attn", kv="bf16", B=64, Hq=64, Hkv=8, q_len=1, groups=1,
             loose=0, pre_lo=128, pre_hi=128, tail_lo=100, tail_hi=2000, lens=2),
        # one GPU out of eight, many samples of a document
        dict(name="shared_document_32k", op="attn", kv="e4m3", B=128, Hq=16, Hkv=2, q_len=1,
             groups=1, loose=0, pre_lo=512, pre_hi=512, tail_lo=16, tail_hi=4096, lens=3),
        # six prompts with eight samples each, a draft token beside the sampled one
        dict(name="shared_block_draft", op="attn", kv="block", B=48, Hq=48, Hkv=8, q_len=2,
             groups=6, loose=0, pre_lo=20, pre_hi=100, tail_lo=50, tail_hi=1500, lens=4),
        # odd groups, odd heads and requests of no group
        dict(name="shared_odd", op="attn", kv="bf16", B=37, Hq=15, Hkv=3, q_len=3, groups=5,
             loose=6, pre_lo=3, pre_hi=90, tail_lo=3, tail_hi=3000, lens=5),
        # a large batch of one head: prompts of three kinds
        dict(name="shared_wide", op="attn", kv="bf16", B=256, Hq=8, Hkv=1, q_len=1, groups=3,
             loose=16, pre_lo=64, pre_hi=256, tail_lo=64, tail_hi=4096, lens=6),
        # eight samples of one prompt begin
        dict(name="fork_samples", op="fork", kv="bf16", parents=1, children=8, Hkv=1, lo=500,
             hi=1000, lens=7),
        # beams: sixteen parents, sixty-four children, block scales
        dict(name="fork_beams", op="fork", kv="block", parents=16, children=64, Hkv=8, lo=1000,
             hi=8000, lens=8),
        # a handful of requests leave, others take their places
        dict(name="turnover_few", op="turn", B=32, rows=4, lo=100, hi=3000, lens=9),
        # a whole batch of long requests is exchanged
        dict(name="turnover_batch", op="turn", B=256, rows=200, lo=1000, hi=32768, lens=10),
        # a small cache with holes
        dict(name="compact_small", op="compact", kv="e4m3", pages=300, Hkv=2, live=0.6, B=20,
             lens=11),
        # a layer's gigabyte, a third of it free
        dict(name="compact_large", op="compact", kv="bf16", pages=4096, Hkv=8, live=0.67, B=100,
             lens=12),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "fork", "turn", "compact"])
    kv = rng.choice(["bf16", "e4m3", "block"])
    Hkv = rng.choice([1, 1, 2, 3, 4, 8])
    lens = rng.randrange(1 << 30)
    if op == "attn":
        q_len = rng.choice([1, 1, 1, 2, 3])
        B = _log(rng, 2, 128 if Hkv < 4 else 64)
        loose = rng.randint(0, B // 4)
        pre_lo = _log(rng, 1, 120)
        tail_lo = _log(rng, q_len, 500)
        G = rng.randint(1, min(16, 64 // Hkv) // q_len)
        return dict(op=op, kv=kv, B=B, Hq=G * Hkv, Hkv=Hkv, q_len=q_len, loose=loose,
                    groups=_log(rng, 1, max(1, (B - loose) // 2)), pre_lo=pre_lo,
                    pre_hi=_log(rng, pre_lo, 130), tail_lo=tail_lo,
                    tail_hi=_log(rng, tail_lo, 2000), lens=lens)
    lo = _log(rng, 1, 2000)
    if op == "fork":
        return dict(op=op, kv=kv, parents=_log(rng, 1, 20), children=_log(rng, 1, 64), Hkv=Hkv,
                    lo=lo, hi=_log(rng, lo, 6000), lens=lens)
    if op == "turn":
        B = _log(rng, 1, 200)
        return dict(op=op, B=B, rows=rng.randint(1, B), lo=lo, hi=_log(rng, lo, 30000), lens=lens)
    return dict(op=op, kv=kv, pages=_log(rng, 50, 2000), Hkv=Hkv,
                live=round(rng.uniform(0.05, 0.95), 2), B=_log(rng, 1, 64), lens=lens)


def _spread(r, lo, hi, n):
    """n whole numbers, log-uniform on [lo, hi]."""
    return [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo), math.log(hi + 1))))))
            for _ in range(n)]


def _groups(case):
    """The groups' first requests (and the end), their shared pages, all lengths."""
    r = random.Random(case["lens"])
    n = case["B"] - case["loose"]
    cuts = sorted(r.sample(range(1, n), case["groups"] - 1)) if case["groups"] > 1 else []
    starts = [0] + cuts + [n]
    pages = _spread(r, case["pre_lo"], case["pre_hi"], case["groups"])
    tails = _spread(r, case["tail_lo"], case["tail_hi"], case["B"])
    lens = list(tails)
    for g, p in enumerate(pages):
        for b in range(starts[g], starts[g + 1]):
            lens[b] += p * PAGE
    return starts, pages, lens


def _page_bytes(case):
    """Bytes of one page of K and V and its scales."""
    return 2 * PAGE * case["Hkv"] * D * (2 if case["kv"] == "bf16" else 1) + \
        (case["Hkv"] * 32 if case["kv"] == "block" else 0)


def _family(case):
    """A fork's parents' lengths, and the old and the new children's parents and lengths."""
    r = random.Random(case["lens"])
    P, n = case["parents"], case["children"]
    have = _spread(r, case["lo"], case["hi"], P)
    born = []
    for _ in range(2):
        src = [r.randrange(P) for _ in range(n)]
        born.append((src, [have[s] if r.random() < 0.5 else r.randint(1, have[s]) for s in src]))
    return have, born[0], born[1]


def _exchange(case):
    """A turnover's rows, all lengths before it, and those rows' lengths after it."""
    r = random.Random(case["lens"])
    before = _spread(r, case["lo"], case["hi"], case["B"])
    rows = r.sample(range(case["B"]), case["rows"])
    return rows, before, _spread(r, case["lo"], case["hi"], case["rows"])


def _pages_of(n):
    return -(-n // PAGE)


def work(case):
    if case["op"] == "attn":
        Hq, Hkv, n = case["Hq"], case["Hkv"], case["q_len"]
        starts, pages, lens = _groups(case)
        members = [starts[g + 1] - starts[g] for g in range(len(pages))]
        tokens = sum(lens) - sum((m - 1) * p * PAGE for m, p in zip(members, pages))
        pairs = sum(max(L - n + 1 + i, 0) for L in lens for i in range(n))
        rows = case["B"] * n * Hq
        bpq = 2 * D if case["kv"] == "bf16" else D + 4
        return {"bytes": tokens * (_page_bytes(case) + 4) / PAGE + rows * (bpq + 2 * D) +
                4 * len(lens), "flops": 4 * D * Hq * pairs}
    if case["op"] == "fork":
        _, old, new = _family(case)
        held = sum(_pages_of(L) for L in old[1]) + sum(_pages_of(L) for L in new[1])
        copied = sum(L % PAGE > 0 for L in new[1])
        # table entries and counts read and written; pages read and written
        return {"bytes": 16 * held + 2 * copied * _page_bytes(case), "flops": 0}
    if case["op"] == "turn":
        rows, before, after = _exchange(case)
        moved = sum(_pages_of(before[b]) for b in rows) + sum(_pages_of(L) for L in after)
        return {"bytes": 20 * moved, "flops": 0}
    live = max(1, int(case["pages"] * case["live"]))
    moved = live * (1 - live / case["pages"])  # (expected: the holes lie at random)
    return {"bytes": 2 * moved * _page_bytes(case) + 16 * case["pages"] + 8 * live, "flops": 0}


# ------------------------------------------------------------------ inputs
def _pow2_scale(a):
    """The smallest power of two s >= 2^-126 with a <= 448 s."""
    m, e = torch.frexp(a.double() / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp_min(-126)
    return ((torch.where(a > 0, e, -126) + 127) << 23).int().view(torch.float32)


def _to_e4m3(x):
    return x.clamp(-448.0, 448.0).to(E4M3)


def _rows(shape, gen, spread):
    """Normal rows whose magnitude varies over tokens and heads, with a few large channels."""
    x = torch.randn(shape, generator=gen, device="cuda")
    size = torch.exp2(torch.rand(shape[:-1], generator=gen, device="cuda") * spread - spread / 2)
    chan = torch.ones(shape[-1], device="cuda")
    chan[::29] = 4.0
    return x * size[..., None] * chan


def _cache(s, kv, total, Hkv, gen):
    """K and V pages with what they are multiplied by."""
    s["ks"] = s["vs"] = 1.0
    s["scale"] = None
    if kv == "block":
        s["scale"] = torch.empty((total, Hkv, 2, PAGE // BLOCK), device="cuda")
    for i, name in enumerate(("k", "v")):
        x = _rows((total, PAGE, Hkv, D), gen, 3.0)
        if kv == "bf16":
            s[name] = x.bfloat16()
        elif kv == "e4m3":
            s[name + "s"] = float(x.abs().max()) / 448.0
            s[name] = _to_e4m3(x / s[name + "s"])
        else:
            f = _pow2_scale(x.view(total, PAGE // BLOCK, BLOCK, Hkv, D).abs().amax((2, 4)))
            s["scale"][:, :, i] = f.transpose(1, 2)
            s[name] = _to_e4m3(x / f.repeat_interleave(BLOCK, 1)[..., None])


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(s, total, perm, taken):
    """A pool whose pages perm[:taken] are held, as s["table"] says."""
    held = s["table"][s["table"] >= 0].long()
    s["refs"] = torch.zeros(total, dtype=torch.int32, device="cuda").index_add_(
        0, held, torch.ones_like(held, dtype=torch.int32))
    s["free"] = torch.zeros(total, dtype=torch.int32, device="cuda")
    s["free"][:total - taken] = perm[taken:]
    s["state"] = _ints([total - taken, 0, 0, 0])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    s = dict(case=case)
    if case["op"] == "attn":
        B, Hq, Hkv, n = case["B"], case["Hq"], case["Hkv"], case["q_len"]
        starts, pages, lens = _groups(case)
        s["starts"], s["pages"], s["lens"] = _ints(starts), _ints(pages), _ints(lens)
        s["T"] = max(lens)
        of = [next((g for g in range(len(pages)) if starts[g] <= b < starts[g + 1]), -1)
              for b in range(B)]
        per = [_pages_of(L) for L in lens]
        skip = [pages[g] if g >= 0 else 0 for g in of]
        total = sum(pages) + sum(p - k for p, k in zip(per, skip))
        perm = torch.randperm(total, generator=gen, device="cuda").int()
        table = torch.full((B, max(per)), -1, dtype=torch.int32, device="cuda")
        at, first = 0, []
        for p in pages:
            first.append(at)
            at += p
        for b in range(B):
            if skip[b]:
                table[b, :skip[b]] = perm[first[of[b]]:first[of[b]] + skip[b]]
            table[b, skip[b]:per[b]] = perm[at:at + per[b] - skip[b]]
            at += per[b] - skip[b]
        s["table"] = table
        _cache(s, case["kv"], total, Hkv, gen)
        q = torch.randn((B, n, Hq, D), generator=gen, device="cuda")
        s["qs"] = None
        if case["kv"] == "bf16":
            s["q"] = q.bfloat16()
        else:
            s["qs"] = q.abs().amax(-1) / 448.0
            s["q"] = _to_e4m3(q / s["qs"][..., None])
        s["out"] = torch.zeros((B, n, Hq, D), dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "fork":
        have, old, new = _family(case)
        P, n = case["parents"], case["children"]
        width = max(_pages_of(L) for L in have)
        total = sum(_pages_of(L) for L in have) + 2 * n + 3
        perm = torch.randperm(total, generator=gen, device="cuda").int()
        table = torch.full((P + n, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, L in enumerate(have):
            table[i, :_pages_of(L)] = perm[at:at + _pages_of(L)]
            at += _pages_of(L)
        for i, (src, L) in enumerate(zip(*old)):
            table[P + i, :L // PAGE] = table[src, :L // PAGE]
            if L % PAGE:
                table[P + i, L // PAGE] = perm[at]
                at += 1
        s["table"] = table
        _pool(s, total, perm, at)
        s["src"], s["len"] = _ints(new[0]), _ints(new[1])
        s["dst"] = _ints(list(range(P, P + n)))
        s["copies"] = torch.zeros((n + 1, 2), dtype=torch.int32, device="cuda")
        _cache(s, case["kv"], total, case["Hkv"], gen)
        return s
    if case["op"] == "turn":
        rows, before, after = _exchange(case)
        per = [_pages_of(L) for L in before]
        total = sum(per) + sum(_pages_of(L) for L in after) + 7
        perm = torch.randperm(total, generator=gen, device="cuda").int()
        table = torch.full((case["B"], _pages_of(max(before + after))), -1, dtype=torch.int32,
                           device="cuda")
        at = 0
        for b, p in enumerate(per):
            table[b, :p] = perm[at:at + p]
            at += p
        s["table"] = table
        _pool(s, total, perm, at)
        s["rows"], s["len"] = _ints(rows), _ints(after)
        return s
    # a fragmented pool: the live pages anywhere, a tenth of them held by two rows
    total, B = case["pages"], case["B"]
    live = max(1, int(total * case["live"]))
    perm = torch.randperm(total, generator=gen, device="cuda").int()
    width = -(-live // B) + 4
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        mine = perm[:live][b::B]
        table[b, :mine.numel()] = mine
        if b % 10 == 1:  # its first pages are those of the row before
            extra = table[b - 1, :min(4, width - mine.numel())]
            table[b, mine.numel():mine.numel() + extra.numel()] = extra
    s["table"] = table
    _pool(s, total, perm, live)
    s["copies"] = torch.zeros((total + 1, 2), dtype=torch.int32, device="cuda")
    s["table_out"] = torch.zeros_like(table)
    s["refs_out"] = torch.zeros_like(s["refs"])
    s["free_out"] = torch.zeros_like(s["free"])
    s["state_out"] = torch.zeros_like(s["state"])
    _cache(s, case["kv"], total, case["Hkv"], gen)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_attention(s):
    """Softmax attention of every request over its whole context."""
    c = s["case"]
    B, Hq, Hkv, n = c["B"], c["Hq"], c["Hkv"], c["q_len"]
    G = Hq // Hkv
    L = s["lens"].long()[:, None]
    j = torch.arange(s["T"], device="cuda").expand(B, s["T"])
    live = j < L
    at = j.minimum(L - 1)
    page = s["table"].long().gather(1, at // PAGE)
    slot = at % PAGE
    K, V = s["k"][page, slot].float(), s["v"][page, slot].float()  # [B, T, Hkv, D]
    if s["scale"] is not None:
        sc = s["scale"].permute(0, 3, 2, 1)[page, slot // BLOCK]  # [B, T, 2, Hkv]
        K, V = K * sc[:, :, 0, :, None], V * sc[:, :, 1, :, None]
    else:
        K, V = K * s["ks"], V * s["vs"]
    q = s["q"].float() if s["qs"] is None else s["q"].float() * s["qs"][..., None]
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, K.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    p = L - n + torch.arange(n, device="cuda")  # the queries' positions [B, n]
    see = (live[:, None, :] & (j[:, None, :] <= p[:, :, None]))[:, None, None]
    x = x.view(B, Hkv, G, n, -1).masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp_(x.sub_(m))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hkv, G * n, -1), V.permute(0, 2, 1, 3)).view(B, Hkv, G, n, D)
    o = torch.where(z > 0, o / z.clamp_min(1e-38), torch.zeros_like(o))
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D))
    return s["out"]


def _plain_free(s, rows):
    """All pages of the rows go back; the first one listed will be the next handed out."""
    held = s["table"][rows]
    pages = held[held >= 0].long()
    s["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    order = torch.arange(pages.numel(), device="cuda")
    first = torch.full((s["refs"].numel(),), pages.numel(), device="cuda").scatter_reduce_(
        0, pages, order, "amin")
    back = pages[(s["refs"][pages] == 0) & (first[pages] == order)].int()
    top = s["state"][0].long()
    s["free"][top + torch.arange(back.numel(), device="cuda")] = back.flip(0)
    s["state"][0] += back.numel()
    s["table"][rows] = -1


def _plain_take(s, want):
    """A page off the stack for each true entry of `want`, in order; -1 for the others."""
    rank = torch.cumsum(want.flatten().long(), 0).view(want.shape)
    page = s["free"][(s["state"][0] - rank).clamp_min(0)]
    page = torch.where(want, page, -1)
    s["refs"][page[want].long()] = 1
    s["state"][0] -= want.sum()
    return page


def _plain_copy(s, src, dst):
    s["k"].view(torch.uint8)[dst] = s["k"].view(torch.uint8)[src]
    s["v"].view(torch.uint8)[dst] = s["v"].view(torch.uint8)[src]
    if s["scale"] is not None:
        s["scale"][dst] = s["scale"][src]


def _plain_fork(s):
    src, dst, n = s["src"].long(), s["dst"].long(), s["len"].long()
    _plain_free(s, dst)
    whole, part = n // PAGE, n % PAGE > 0
    j = torch.arange(s["table"].shape[1], device="cuda")
    shared = torch.where(j < whole[:, None], s["table"][src], -1)
    pages = shared[shared >= 0].long()
    s["refs"].index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    fresh = _plain_take(s, part)
    s["table"][dst] = torch.where((j == whole[:, None]) & part[:, None], fresh[:, None], shared)
    a, b = s["table"][src[part], whole[part]], fresh[part]
    s["copies"][0, 0], s["copies"][0, 1] = a.numel(), 0
    s["copies"][1:1 + a.numel()] = torch.stack([a, b], 1)
    _plain_copy(s, a.long(), b.long())
    return _forked(s)


def _forked(s):
    out = [s["table"], s["refs"], s["free"], s["state"], s["copies"], s["k"], s["v"]]
    return out if s["scale"] is None else out + [s["scale"]]


def _plain_turn(s):
    rows = s["rows"].long()
    _plain_free(s, rows)
    j = torch.arange(s["table"].shape[1], device="cuda")
    s["table"][rows] = _plain_take(s, j < ((s["len"].long() + PAGE - 1) // PAGE)[:, None])
    return [s["table"], s["refs"], s["free"], s["state"]]


def _plain_compact(s):
    """The live pages behind the first `live` places move, in order, into the holes there."""
    refs, total = s["refs"], s["refs"].numel()
    at = torch.arange(total, device="cuda")
    live = (refs > 0).sum()
    src, dst = at[(refs > 0) & (at >= live)], at[(refs == 0) & (at < live)]
    to = at.clone()
    to[src] = dst
    s["table_out"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp_min(0).long()],
                                     s["table"].long()))
    s["refs_out"].copy_(torch.where(at < live, refs, torch.zeros_like(refs)))
    s["refs_out"][dst] = refs[src]
    s["free_out"].copy_(torch.where(at < total - live, total - 1 - at, s["free_out"].long()))
    s["state_out"].copy_(s["state"])
    s["state_out"][0] = total - live
    s["copies"][0, 0], s["copies"][0, 1] = src.numel(), 0
    s["copies"][1:1 + src.numel()] = torch.stack([src, dst], 1).int()
    _plain_copy(s, src, dst)
    return _compacted(s)


def _compacted(s):
    out = [s["table_out"], s["refs_out"], s["free_out"], s["state_out"], s["copies"], s["k"],
           s["v"]]
    return out if s["scale"] is None else out + [s["scale"]]


# ------------------------------------------------------------------ the pass
def run(s):
    c = s["case"]
    if not own:
        return {"attn": _plain_attention, "fork": _plain_fork, "turn": _plain_turn,
                "compact": _plain_compact}[c["op"]](s)
    import load_balanced_paged_assign_gb300 as hd
    if c["op"] == "attn":
        ws = s.get("ws")
        if ws is None:
            dtype = {"bf16": hd.HPC_KV_BF16, "e4m3": hd.HPC_KV_FP8_E4M3,
                     "block": hd.HPC_KV_E4M3_BLOCK}[c["kv"]]
            ws = s["ws"] = hd.SharedWorkspace(c["B"], c["Hq"], c["Hkv"], c["groups"],
                                              kv_dtype=dtype, q_len=c["q_len"])
        hd.hpc_decode_step_shared(s["q"], s["qs"], s["k"], s["v"], s["ks"], s["vs"], s["scale"],
                                  s["table"], s["lens"], s["starts"], s["pages"], c["Hq"],
                                  c["Hkv"], c["q_len"], 1.0 / math.sqrt(D), 2, ws, s["out"])
        return s["out"]
    pool = s.get("pool")
    if pool is None:
        pool = s["pool"] = hd.PagePool.of(s["refs"], s["free"], s["state"])
    if c["op"] == "fork":
        hd.hpc_kv_free(pool, s["table"], s["dst"])
        hd.hpc_kv_fork(pool, s["table"], s["src"], s["dst"], s["len"], s["copies"])
        hd.hpc_kv_copy_pages(s["copies"], s["k"], s["v"], s["scale"])
        return _forked(s)
    if c["op"] == "turn":
        hd.hpc_kv_free(pool, s["table"], s["rows"])
        hd.hpc_kv_extend(pool, s["table"], s["rows"], s["len"])
        return [s["table"], s["refs"], s["free"], s["state"]]
    to = s.get("pool_out")
    if to is None:
        to = s["pool_out"] = hd.PagePool.of(s["refs_out"], s["free_out"], s["state_out"])
    hd.hpc_kv_compact(pool, s["table"], s["copies"], s["table_out"], to)
    hd.hpc_kv_copy_pages(s["copies"], s["k"], s["v"], s["scale"])
    return _compacted(s)


# ------------------------------------------------------------------ 64 bits
def _exact_attention(s):
    c = s["case"]
    n, G = c["q_len"], c["Hq"] // c["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :_pages_of(L)].long()
        kv = []
        for i, name in enumerate(("k", "v")):
            x = s[name][pages].double()
            if s["scale"] is not None:
                f = s["scale"][pages][:, :, i].double()  # [P, Hkv, 4]
                x = x * f.repeat_interleave(BLOCK, 2).transpose(1, 2)[..., None]
            else:
                x = x * s[name + "s"]
            kv.append(x.reshape(-1, c["Hkv"], D)[:L])
        hide = torch.arange(L, device="cuda") > (L - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(c["Hkv"]):
            q = s["q"][b, :, h * G:(h + 1) * G].double()
            if s["qs"] is not None:
                q = q * s["qs"][b, :, h * G:(h + 1) * G].double()[..., None]
            x = torch.einsum("igd,td->git", q, kv[0][:, h]) / math.sqrt(D)
            w = torch.nan_to_num(torch.softmax(x.masked_fill(hide, -math.inf), -1), nan=0.0)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("git,td->igd", w, kv[1][:, h])
    return out


def _listed_pool(s):
    """The table and the pool as Python lists."""
    return (s["table"].tolist(), s["refs"].tolist(), s["free"].tolist(), s["state"].tolist())


def _give_back(table, refs, free, state, rows):
    back = []
    for r in rows:
        for j, p in enumerate(table[r]):
            if p >= 0:
                refs[p] -= 1
                back.append(p)
                table[r][j] = -1
    seen = set()
    back = [p for p in back if refs[p] == 0 and not (p in seen or seen.add(p))]
    for i, p in enumerate(reversed(back)):
        free[state[0] + i] = p
    state[0] += len(back)


def _hand_out(refs, free, state):
    state[0] -= 1
    refs[free[state[0]]] = 1
    return free[state[0]]


def _moved(s, pairs):
    """The caches after the copies, as 64-bit numbers."""
    out = []
    for name in ("k", "v", "scale"):
        if s[name] is not None:
            x = s[name].double()
            if pairs:
                x[[b for _, b in pairs]] = x[[a for a, _ in pairs]]
            out.append(x)
    return out


def _exact_pages(s):
    op = s["case"]["op"]
    table, refs, free, state = _listed_pool(s)
    if op == "turn":
        rows = s["rows"].tolist()
        _give_back(table, refs, free, state, rows)
        for r, L in zip(rows, s["len"].tolist()):
            for j in range(_pages_of(L)):
                table[r][j] = _hand_out(refs, free, state)
        return [_ints(x) for x in (table, refs, free, state)]
    pairs = []
    if op == "fork":
        dst = s["dst"].tolist()
        _give_back(table, refs, free, state, dst)
        for a, b, L in zip(s["src"].tolist(), dst, s["len"].tolist()):
            for j in range(L // PAGE):
                table[b][j] = table[a][j]
                refs[table[a][j]] += 1
            if L % PAGE:
                table[b][L // PAGE] = _hand_out(refs, free, state)
                pairs.append((table[a][L // PAGE], table[b][L // PAGE]))
    else:
        live = sum(r > 0 for r in refs)
        holes = [p for p in range(live) if refs[p] == 0]
        pairs = list(zip([p for p in range(live, len(refs)) if refs[p] > 0], holes))
        to = dict(pairs)
        table = [[to.get(p, p) for p in row] for row in table]
        for a, b in pairs:
            refs[b], refs[a] = refs[a], 0
        state[0] = len(refs) - live
        free = list(range(len(refs) - 1, live - 1, -1)) + [0] * live
    copies = [[len(pairs), 0]] + [list(p) for p in pairs]
    copies += [[0, 0]] * (s["copies"].shape[0] - len(copies))
    return [_ints(x) for x in (table, refs, free, state, copies)] + _moved(s, pairs)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] == "attn" else _exact_pages(s)
