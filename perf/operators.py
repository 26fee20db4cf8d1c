"""The 8-bit cache with block scales and windowed attention, as measured.

Every case is one pass through an operator of a serving step: a decode step
over a paged cache (the whole context or a window with sinks; BF16, E4M3 with
one scale per cache, or E4M3 with one scale for each 16 tokens and head), a
prompt's attention with a window, or the prologue that writes new tokens into
the block-scaled cache followed by the read-back of those tokens as BF16.

`run` computes the operator in plain torch operations (32 bits, rounded once
at the end) where `own` is false, and calls the framework where it is true.
Caches are [pages, 64, Hkv, 128]; block scales [pages, Hkv, 2, 4] hold K's
four scales of a page and then V's.
"""

import math
import random

import torch

own = False

D = 128
PAGE = 64
BLOCK = 16
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
ROPE_BASE = 1e6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's short chat, the latency of a single small decode step
        dict(name="block_decode_1x1k", op="decode", kv="block", B=1, Hq=8, Hkv=1, q_len=1,
             window=0, sinks=0, lo=1000, hi=1000, lens=1),
        # a mixed batch of one GPU out of eight: log-uniform contexts up to 128K
        dict(name="block_decode_mixed_128k", op="decode", kv="block", B=64, Hq=8, Hkv=1, q_len=1,
             window=0, sinks=0, lo=1024, hi=131072, lens=2),
        # all heads on one GPU, one draft token beside the sampled one
        dict(name="block_decode_draft", op="decode", kv="block", B=64, Hq=64, Hkv=8, q_len=2,
             window=0, sinks=0, lo=512, hi=16384, lens=3),
        # a few users on a window layer, odd window and sinks
        dict(name="window_decode_small", op="decode", kv="bf16", B=4, Hq=8, Hkv=1, q_len=1,
             window=500, sinks=5, lo=300, hi=4000, lens=4),
        # a full batch on a window layer, contexts both below and far beyond the window
        dict(name="window_decode_bf16", op="decode", kv="bf16", B=64, Hq=64, Hkv=8, q_len=1,
             window=4096, sinks=64, lo=1024, hi=16384, lens=5),
        # long contexts over a short window, one scale per cache
        dict(name="window_decode_e4m3", op="decode", kv="e4m3", B=128, Hq=16, Hkv=2, q_len=1,
             window=1024, sinks=16, lo=1024, hi=32768, lens=6),
        # block scales and window together, a draft token, six query heads for each KV head
        dict(name="window_decode_block_draft", op="decode", kv="block", B=48, Hq=48, Hkv=8,
             q_len=2, window=2048, sinks=4, lo=500, hi=16384, lens=7),
        # a short prompt on a layer with a small window
        dict(name="window_prefill_q512", op="prefill", B=1, Hq=64, Hkv=8, q_len=512, prefix=0,
             window=128, sinks=4),
        # a long prompt
        dict(name="window_prefill_q8k", op="prefill", B=1, Hq=64, Hkv=8, q_len=8192, prefix=0,
             window=1024, sinks=64),
        # two chunks behind a cached prefix, odd sizes
        dict(name="window_extend_2q1k", op="prefill", B=2, Hq=64, Hkv=8, q_len=1000, prefix=3111,
             window=2000, sinks=10),
        # the new token of every request of a decode step, FP8 queries
        dict(name="write_decode", op="write", B=64, new=1, lo=1024, hi=8192, lens=11, Hq=8,
             Hkv=1, interleaved=False, q8=True),
        # an 8K-token prompt, BF16 queries for the prefill attention
        dict(name="write_prompt_8k", op="write", B=1, new=8192, lo=0, hi=0, lens=12, Hq=64,
             Hkv=8, interleaved=False, q8=False),
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prefill", "write"])
    Hkv = rng.choice([1, 1, 2, 4, 8])
    if op == "decode":
        q_len = rng.choice([1, 1, 1, 2, 3])
        G = rng.randint(1, 16 // q_len)
        lo = _log(rng, 1, 2000)
        hi = _log(rng, lo, 16384)
        kv = rng.choice(["block", "block", "bf16", "e4m3"])
        window = _log(rng, 1, 8192) if kv != "block" or rng.random() < 0.5 else 0
        return dict(op=op, kv=kv, B=_log(rng, 1, 64), Hq=G * Hkv, Hkv=Hkv, q_len=q_len,
                    window=window, sinks=_log(rng, 1, 300) - 1 if window else 0, lo=lo, hi=hi,
                    lens=rng.randrange(1 << 30))
    if op == "prefill":
        return dict(op=op, B=rng.randint(1, 3), Hq=rng.choice([1, 2, 4, 8]) * Hkv, Hkv=Hkv,
                    q_len=_log(rng, 1, 2048), prefix=_log(rng, 1, 4096) - 1,
                    window=_log(rng, 1, 4096), sinks=_log(rng, 1, 300) - 1)
    new = _log(rng, 1, 2048)
    return dict(op=op, B=_log(rng, 1, max(1, 4096 // new)), new=new, lo=0, hi=_log(rng, 1, 4096),
                lens=rng.randrange(1 << 30), Hq=rng.choice([1, 4, 8]) * Hkv, Hkv=Hkv,
                interleaved=rng.random() < 0.5, q8=rng.random() < 0.5)


def _lengths(case):
    """Live tokens of each request, log-uniform on [lo, hi] (for a write: those before it)."""
    if case["op"] == "prefill":
        return [case["prefix"] + case["q_len"]] * case["B"]
    r = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    return [min(hi, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 2)))) - 1)
            if hi > lo else lo for _ in range(case["B"])]


def _visible(p, window, sinks):
    """Tokens that a query at position p sees."""
    if p < 0:
        return 0
    return p + 1 if not window else min(p + 1, window + min(sinks, max(p + 1 - window, 0)))


def _touched(L, q_len, window, sinks):
    """Tokens that some query of a request of L tokens sees."""
    first = max(0, L - q_len + 1 - window) if window else 0
    return L - first + min(sinks, first)


def work(case):
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "write":
        n = case["B"] * case["new"]
        blocks = case["B"] * (-(-case["new"] // BLOCK))
        q = n * Hq * (D + 4 if case["q8"] else 2 * D)
        wrote = n * 2 * Hkv * D + blocks * Hkv * 8
        read_back = wrote + n * 2 * Hkv * 2 * D
        return {"bytes": n * ((Hq + 2 * Hkv) * 2 * D + 8) + q + wrote + read_back,
                "flops": n * (Hq + Hkv) * D * 10}
    q_len, W, S = case["q_len"], case["window"], case["sinks"]
    kv = case.get("kv", "bf16")
    per_token = 2 * Hkv * {"bf16": 2 * D, "e4m3": D, "block": D + 4 / BLOCK}[kv]
    rows = case["B"] * q_len * Hq
    lens = _lengths(case)
    tokens = sum(_touched(L, q_len, W, S) for L in lens)
    pairs = sum(_visible(L - q_len + i, W, S) for L in lens[:1] for i in range(q_len)) * len(lens) \
        if case["op"] == "prefill" else \
        sum(_visible(L - q_len + i, W, S) for L in lens for i in range(q_len))
    bpq = 2 * D if kv == "bf16" else D + 4
    return {"bytes": tokens * (per_token + 4 / PAGE) + rows * (bpq + 2 * D) + 4 * len(lens),
            "flops": 4 * D * Hq * pairs}


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


def _pages(lens, gen):
    """A block table that hands a random permutation of the pages to the requests."""
    per = [-(-L // PAGE) for L in lens]
    total = max(sum(per), 1)
    perm = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(per):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, total


def _block_cache(total, Hkv, gen):
    """Codes and block scales of a cache of K and V rows."""
    scale = torch.empty((total, Hkv, 2, PAGE // BLOCK), device="cuda")
    out = []
    for i in range(2):
        x = _rows((total, PAGE, Hkv, D), gen, 3.0)
        s = _pow2_scale(x.view(total, PAGE // BLOCK, BLOCK, Hkv, D).abs().amax((2, 4)))
        scale[:, :, i] = s.transpose(1, 2)
        s = s.repeat_interleave(BLOCK, 1)
        out.append(_to_e4m3(x / s[..., None]))
    return out[0], out[1], scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    Hq, Hkv, B = case["Hq"], case["Hkv"], case["B"]
    s = dict(case=case)
    if case["op"] == "write":
        before = _lengths(case)
        lens = [L + case["new"] for L in before]
        s["table"], total = _pages(lens, gen)
        s["k"], s["v"], s["scale"] = _block_cache(total, Hkv, gen)
        n = B * case["new"]
        s["qkv"] = _rows((n, Hq + 2 * Hkv, D), gen, 4.0).bfloat16().view(n, -1)
        s["wq"] = (1 + 0.25 * torch.randn(D, generator=gen, device="cuda")).bfloat16()
        s["wk"] = (1 + 0.25 * torch.randn(D, generator=gen, device="cuda")).bfloat16()
        start = torch.tensor(before, dtype=torch.int32, device="cuda")
        s["start"], s["lens"] = start, start + case["new"]
        s["req"] = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(case["new"])
        s["pos"] = (start[:, None] + torch.arange(case["new"], dtype=torch.int32,
                                                  device="cuda")).reshape(-1).contiguous()
        i = torch.arange(64, dtype=torch.float64, device="cuda")
        s["freq"] = ROPE_BASE ** (-2.0 * i / D)  # the table that a model keeps
        s["q"] = torch.zeros((n, Hq, D), dtype=E4M3 if case["q8"] else torch.bfloat16,
                             device="cuda")
        s["qs"] = torch.zeros((n, Hq), device="cuda") if case["q8"] else None
        # the pages that the prompt's attention reads, in the same order as the cache's
        s["k_out"] = torch.zeros((total, PAGE, Hkv, D), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    lens = _lengths(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"], total = _pages(lens, gen)
    s["T"] = max(max(lens), 1)
    kv = case.get("kv", "bf16")
    s["ks"] = s["vs"] = 1.0
    s["scale"] = None
    if kv == "block":
        s["k"], s["v"], s["scale"] = _block_cache(total, Hkv, gen)
    else:
        s["k"] = _rows((total, PAGE, Hkv, D), gen, 3.0)
        s["v"] = _rows((total, PAGE, Hkv, D), gen, 3.0)
        if kv == "e4m3":
            s["ks"] = float(s["k"].abs().max()) / 448.0
            s["vs"] = float(s["v"].abs().max()) / 448.0
            s["k"], s["v"] = _to_e4m3(s["k"] / s["ks"]), _to_e4m3(s["v"] / s["vs"])
        else:
            s["k"], s["v"] = s["k"].bfloat16(), s["v"].bfloat16()
    q = torch.randn((B, case["q_len"], Hq, D), generator=gen, device="cuda")
    s["qs"] = None
    if kv == "bf16":
        s["q"] = q.bfloat16()
    else:
        s["qs"] = q.abs().amax(-1) / 448.0
        s["q"] = _to_e4m3(q / s["qs"][..., None])
    s["out"] = torch.zeros((B, case["q_len"], Hq, D), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, n = c["B"], c["Hq"], c["Hkv"], c["q_len"]
    G, W, S = Hq // Hkv, c["window"], c["sinks"]
    L = s["lens"].long()[:, None]
    if W and c["op"] == "decode":  # the sinks, then the tokens that some query's window holds
        last = L - (W + n - 1) + torch.arange(W + n - 1, device="cuda")
        first = torch.arange(S, device="cuda").expand(B, S)
        last = torch.where(last >= S, last, -1)
        j = torch.cat([first, last], 1)
    else:
        j = torch.arange(s["T"], device="cuda").expand(B, s["T"])
    live = (j >= 0) & (j < L)
    at = j.clamp(min=0).minimum((L - 1).clamp(min=0))
    page = s["table"].long().gather(1, at // PAGE).clamp(min=0)
    slot = at % PAGE
    K, V = s["k"][page, slot].float(), s["v"][page, slot].float()  # [B, T, Hkv, D]
    if s["scale"] is not None:
        sc = s["scale"].permute(0, 3, 2, 1)[page, slot // BLOCK]  # [B, T, 2, Hkv]
        K, V = K * sc[:, :, 0, :, None], V * sc[:, :, 1, :, None]
    else:
        K, V = K * s["ks"], V * s["vs"]
    V = V * live[:, :, None, None]
    q = s["q"].float() if s["qs"] is None else s["q"].float() * s["qs"][..., None]
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    x = torch.matmul(q, K.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    p = L - n + torch.arange(n, device="cuda")  # the queries' positions [B, n]
    see = live[:, None, :] & (j[:, None, :] <= p[:, :, None])
    if W:
        see &= (j[:, None, :] > p[:, :, None] - W) | (j[:, None, :] < S)
    see = see[:, None, None]  # [B, 1, 1, n, T]
    x = x.view(B, Hkv, G, n, -1).masked_fill_(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp_(x.sub_(m))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hkv, G * n, -1), V.permute(0, 2, 1, 3)).view(B, Hkv, G, n, D)
    o = torch.where(z > 0, o / z.clamp_min(1e-38), torch.zeros_like(o))
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D))
    return s["out"]


def _plain_norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_rope(x, pos, interleaved):
    i = torch.arange(64, dtype=torch.float64, device="cuda")
    a = pos.double()[:, None] * ROPE_BASE ** (-2.0 * i / D)
    c, n = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    y = torch.empty_like(x)
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :64], x[..., 64:])
    if interleaved:
        y[..., 0::2], y[..., 1::2] = u * c - v * n, v * c + u * n
    else:
        y[..., :64], y[..., 64:] = u * c - v * n, v * c + u * n
    return y


def _plain_write(s):
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    pos, req = s["pos"].long(), s["req"].long()
    x = s["qkv"].float().view(-1, Hq + 2 * Hkv, D)
    q = _plain_rope(_plain_norm(x[:, :Hq], s["wq"]), pos, c["interleaved"])
    k = _plain_rope(_plain_norm(x[:, Hq:Hq + Hkv], s["wk"]), pos, c["interleaved"])
    new = torch.stack([k, x[:, Hq + Hkv:]], 2)  # [N, Hkv, 2, D]
    if c["q8"]:
        a = q.abs().amax(-1)
        s["qs"].copy_(torch.where(a > 0, a / 448.0, torch.ones_like(a)))
        s["q"].copy_(_to_e4m3(q / s["qs"][..., None]))
    else:
        s["q"].copy_(q)
    page, slot = s["table"].long()[req, pos // PAGE], pos % PAGE
    block, to = torch.unique(page * (PAGE // BLOCK) + slot // BLOCK, return_inverse=True)
    U = block.numel()
    amax = torch.zeros((U, Hkv, 2), device="cuda").index_reduce_(0, to, new.abs().amax(-1),
                                                                 "amax", include_self=True)
    first = torch.full((U,), BLOCK, device="cuda").scatter_reduce_(0, to, slot % BLOCK, "amin")
    scales = s["scale"].permute(0, 3, 1, 2)  # [pages, 4, Hkv, 2]
    bp, bb = block // (PAGE // BLOCK), block % (PAGE // BLOCK)
    old = scales[bp, bb]
    sc = torch.where((first == 0)[:, None, None], _pow2_scale(amax),
                     torch.maximum(old, _pow2_scale(amax)))
    # tokens that the grown blocks held before: their codes at the new scale
    ratio = torch.where((first == 0)[:, None, None], torch.ones_like(old), old / sc)
    at = bb[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    for i, name in enumerate(("k", "v")):
        cache = s[name].view(torch.uint8)
        held = s[name][bp[:, None], at].float() * ratio[:, None, :, i, None]
        cache[bp[:, None], at] = _to_e4m3(held).view(torch.uint8)
        cache[page, slot] = _to_e4m3(new[:, :, i] / sc[to][:, :, i, None]).view(torch.uint8)
    scales[bp, bb] = sc
    for i, name in enumerate(("k", "v")):  # read back
        r = s[name][page, slot].float() * scales[page, slot // BLOCK][:, :, i, None]
        s[name + "_out"][page, slot] = r.bfloat16()
    return [s["q"], s["qs"], s["k_out"], s["v_out"]]


# ------------------------------------------------------------------ the pass
def run(s):
    c = s["case"]
    if not own:
        return _plain_write(s) if c["op"] == "write" else _plain_attention(s)
    import load_balanced_paged_assign_gb300 as hd
    Hq, Hkv = c["Hq"], c["Hkv"]
    if c["op"] == "write":
        hd.hpc_rope_norm_block(
            s["qkv"], s["wq"], s["wk"], s["pos"], s["req"], Hq, Hkv, s["table"], s["k"], s["v"],
            s["scale"], s["q"], s["qs"], eps=EPS, rope_base=ROPE_BASE,
            rope_layout=hd.HPC_ROPE_INTERLEAVED if c["interleaved"] else hd.HPC_ROPE_HALVES,
            norm_first=True, freq=s["freq"])
        hd.hpc_kv_read_block(s["k"], s["v"], s["scale"], s["table"], s["start"], s["lens"], Hkv,
                             s["k_out"], s["v_out"], s["table"])
        return [s["q"], s["qs"], s["k_out"], s["v_out"]]
    scale = 1.0 / math.sqrt(D)
    if c["op"] == "prefill":
        hd.hpc_prefill_attn_win(s["q"], s["k"], s["v"], s["table"], s["lens"], Hq, Hkv,
                                c["q_len"], c["window"], c["sinks"], scale, s["out"])
        return s["out"]
    ws = s.get("ws")
    if ws is None:
        dtype = {"bf16": hd.HPC_KV_BF16, "e4m3": hd.HPC_KV_FP8_E4M3,
                 "block": hd.HPC_KV_E4M3_BLOCK}[c["kv"]]
        ws = s["ws"] = hd.Workspace(c["B"], Hq, Hkv, kv_dtype=dtype, q_len=c["q_len"])
    hd.hpc_decode_step_win(s["q"], s["qs"], s["k"], s["v"], s["ks"], s["vs"], s["scale"],
                           s["table"], s["lens"], Hq, Hkv, c["q_len"], c["window"], c["sinks"],
                           scale, ws.num_ctas, 2, ws.tmap, ws.part_o, ws.part_lse, s["out"],
                           unit_done=ws.unit_done)
    return s["out"]


# ------------------------------------------------------------------ 64 bits
def _exact_values(s, name, i, pages):
    """The numbers that the cache's pages hold, [tokens, Hkv, D] in 64 bits."""
    x = s[name][pages].double()
    if s["scale"] is not None:
        f = s["scale"][pages][:, :, i].double()  # [P, Hkv, 4]
        x = x * f.repeat_interleave(BLOCK, 2).transpose(1, 2)[..., None]
    else:
        x = x * s["ks" if i == 0 else "vs"]
    return x.reshape(-1, x.shape[2], D)


def _exact_attention(s):
    c = s["case"]
    n, G, W, S = c["q_len"], c["Hq"] // c["Hkv"], c["window"], c["sinks"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        pages = s["table"][b, :-(-L // PAGE)].long()
        K, V = (_exact_values(s, name, i, pages)[:L] for i, name in enumerate("kv"))
        j = torch.arange(L, device="cuda")
        p = (L - n + torch.arange(n, device="cuda"))[:, None]
        hide = j > p
        if W:
            hide |= (j <= p - W) & (j >= S)
        for h in range(c["Hq"]):
            q = s["q"][b, :, h].double()
            if s["qs"] is not None:
                q = q * s["qs"][b, :, h].double()[:, None]
            x = (q @ K[:, h // G].T / math.sqrt(D)).masked_fill(hide, -math.inf)
            w = torch.softmax(x, -1)  # a row that sees nothing comes out as NaN: zero
            out[b, :, h] = torch.nan_to_num(w, nan=0.0) @ V[:, h // G]
    return out


def _exact_pow2(e):
    """2^e in 64 bits, from its exponent field (a power function may be off in the last bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round(y):
    """64-bit numbers within +-448 to the nearest E4M3 value, ties to even."""
    e = torch.frexp(y)[1].clamp_min(-5)  # |y| < 2^e; the smallest normal is 2^-6
    step = _exact_pow2(e - 4)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_write(s):
    c = s["case"]
    Hq, Hkv, new = c["Hq"], c["Hkv"], c["new"]
    x = s["qkv"].double().view(-1, Hq + 2 * Hkv, D)
    pos = s["pos"].double()
    a = pos[:, None] * torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device="cuda"),
                                 -torch.arange(0, D, 2, device="cuda").double() / D)
    turn = torch.polar(torch.ones_like(a), a)[:, None]
    qk = x[:, :Hq + Hkv]
    qk = qk / torch.sqrt(qk.square().mean(-1, keepdim=True) + EPS)
    qk[:, :Hq] *= s["wq"].double()
    qk[:, Hq:] *= s["wk"].double()
    if c["interleaved"]:
        z = torch.complex(qk[..., 0::2].contiguous(), qk[..., 1::2].contiguous()) * turn
        qk = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(qk[..., :64].contiguous(), qk[..., 64:].contiguous()) * turn
        qk = torch.cat([z.real, z.imag], -1)
    rows = [qk[:, Hq:], x[:, Hq + Hkv:]]
    outs = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    table, start = s["table"].tolist(), s["start"].tolist()
    for b in range(c["B"]):
        t, end = start[b], start[b] + new
        while t < end:
            to = min(end, t - t % BLOCK + BLOCK)
            page, blk, r = table[b][t // PAGE], t % PAGE // BLOCK, b * new + t - start[b]
            for i in range(2):
                y = rows[i][r:r + to - t]
                m = (y.abs().amax((0, 2)) / 448.0).clamp_min(2.0 ** -126)  # [Hkv]
                f, e = torch.frexp(m)
                sc = _exact_pow2(torch.where(f == 0.5, e - 1, e))
                if t % BLOCK:
                    sc = torch.maximum(sc, s["scale"][page, :, i, blk].double())
                outs[i][page, t % PAGE:t % PAGE + to - t] = _exact_round(y / sc[:, None]) * \
                    sc[:, None]
            t = to
    q = qk[:, :Hq]
    if not c["q8"]:
        return [q, None, outs[0], outs[1]]
    big = q.abs().amax(-1) / 448.0
    return [_exact_round(q / big[..., None]), big, outs[0], outs[1]]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_write(s) if case["op"] == "write" else _exact_attention(s)
