"""Host-side refusals of the windowed and block-scaled entry points (no GPU:
fake, never-dereferenced device pointers, and CPU tensors for the binding)."""

import ctypes

import pytest
import torch

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as E

FAKE = 0x10000


@pytest.fixture(scope="module", autouse=True)
def built():
    from load_balanced_paged_assign_gb300 import _build
    _build.build()


def fake_map(B=4, Hkv=1, ctas=132, persistent=1):
    m = E.hpc_task_map(FAKE, FAKE, FAKE, FAKE, FAKE, 200, 200, 64, B, Hkv, ctas, persistent, 2, 32)
    return m


def plan(q_len=1, window=100, sinks=4, max_pages=32, B=4, Hkv=1, dtype=0, seqlens=FAKE, m=None):
    m = m or fake_map()
    return hd.lib().hpc_decode_plan_win(seqlens, B, Hkv, max_pages, 132, 2, dtype, q_len, window,
                                        sinks, ctypes.byref(m), None)


def test_plan_refusals():
    assert plan(q_len=0) == E.HPC_ERR_ARG
    assert plan(q_len=17) == E.HPC_ERR_UNSUPPORTED
    assert plan(window=-1) == E.HPC_ERR_ARG
    assert plan(sinks=-1) == E.HPC_ERR_ARG
    assert plan(window=0, sinks=1) == E.HPC_ERR_ARG  # sinks without a window
    assert plan(window=1 << 30) == E.HPC_ERR_UNSUPPORTED
    assert plan(sinks=1 << 30) == E.HPC_ERR_UNSUPPORTED
    assert plan(max_pages=1 << 24) == E.HPC_ERR_UNSUPPORTED  # token indices past 2^30
    assert plan(seqlens=None) == E.HPC_ERR_ARG
    assert plan(B=70) == E.HPC_ERR_WORKSPACE
    assert plan(dtype=3) == E.HPC_ERR_ARG
    # descriptors of head pairs: room for 2 num_ctas + B Hkv
    assert plan(B=4, Hkv=2, dtype=1) == E.HPC_ERR_WORKSPACE
    assert plan(B=4, Hkv=2, dtype=2, window=0, sinks=0) == E.HPC_ERR_WORKSPACE


def attn(step=False, q=FAKE, qs=None, k=FAKE, v=FAKE, num_pages=10, kvs=None, dtype=0, bt=FAKE,
         max_pages=4, B=4, Hq=8, Hkv=1, D=128, q_len=1, window=0, sinks=0, sm=0.088, po=FAKE,
         done=FAKE, out=FAKE, m=None):
    m = m or fake_map()
    head = [q, qs, k, v, num_pages, 1.0, 1.0, kvs, dtype, bt, max_pages, FAKE, B, Hq, Hkv, D,
            q_len, window, sinks, sm]
    L = hd.lib()
    if step:
        return L.hpc_decode_step_win(*head, 132, 2, ctypes.byref(m), po, FAKE, done, out, None)
    return L.hpc_decode_attn_win(*head, ctypes.byref(m), po, FAKE, done, out, None)


@pytest.mark.parametrize("step", [False, True])
def test_attention_refusals(step):
    ARG, UNS = E.HPC_ERR_ARG, E.HPC_ERR_UNSUPPORTED
    assert attn(step, D=64) == UNS
    assert attn(step, Hq=17) == UNS
    assert attn(step, Hq=6, Hkv=4) == UNS
    assert attn(step, q_len=0) == ARG
    assert attn(step, q_len=3) == UNS  # 24 query rows per KV head
    assert attn(step, q_len=1 << 29) == UNS
    assert attn(step, window=-5) == ARG
    assert attn(step, sinks=2) == ARG
    assert attn(step, window=8, sinks=-1) == ARG
    assert attn(step, max_pages=1 << 24, B=1) == UNS
    assert attn(step, dtype=2) == ARG  # block-scaled without scales
    assert attn(step, dtype=1, qs=FAKE, kvs=FAKE) == ARG  # scales for another cache type
    assert attn(step, kvs=FAKE) == ARG


def test_attention_refusals_of_pointers_and_maps():
    ARG = E.HPC_ERR_ARG
    assert attn(dtype=9) == ARG
    assert attn(dtype=2, kvs=FAKE, qs=None) == ARG  # E4M3 queries need their scales
    assert attn(dtype=2, kvs=FAKE + 4, qs=FAKE) == ARG
    assert attn(q=FAKE + 8) == ARG
    assert attn(k=None) == ARG
    assert attn(num_pages=0) == ARG
    assert attn(sm=float("nan")) == ARG
    assert attn(done=None) == ARG and attn(out=None) == ARG  # both or neither
    assert attn(m=fake_map(B=5)) == ARG
    # a map planned without this window, and one with a window for a plain call
    assert attn(window=100, sinks=4) == ARG
    assert attn(m=fake_map(persistent=1 | (77 << 1))) == ARG
    assert attn(window=100, m=fake_map(persistent=0)) == ARG  # a static map has no window
    m = fake_map(persistent=1 | (77 << 1))
    assert hd.lib().hpc_decode_attn(FAKE, None, FAKE, FAKE, 10, 1.0, 1.0, 0, FAKE, 4, FAKE, 4, 8,
                                    1, 128, 0.088, ctypes.byref(m), FAKE, FAKE, None) == ARG
    # the calls without block scales do not take the block-scaled type
    m = fake_map()
    assert hd.lib().hpc_decode_attn(FAKE, FAKE, FAKE, FAKE, 10, 1.0, 1.0, 2, FAKE, 4, FAKE, 4, 8,
                                    1, 128, 0.088, ctypes.byref(m), FAKE, FAKE, None) == ARG


def test_prefill_refusals():
    def call(q=FAKE, window=128, sinks=4, q_len=300, D=128, Hq=8, B=2, sm=0.088, out=FAKE,
             max_pages=8):
        return hd.lib().hpc_prefill_attn_win(q, FAKE, FAKE, 100, FAKE, max_pages, FAKE, B, Hq, 2,
                                             D, q_len, window, sinks, sm, out, None, None)

    ARG, UNS = E.HPC_ERR_ARG, E.HPC_ERR_UNSUPPORTED
    assert call(B=0) == E.HPC_OK
    assert call(window=-1) == ARG and call(sinks=-1) == ARG
    assert call(window=0, sinks=3) == ARG
    assert call(window=1 << 30) == UNS and call(sinks=1 << 30) == UNS
    assert call(q_len=0) == ARG
    assert call(D=64) == UNS and call(Hq=7) == UNS
    assert call(q=FAKE + 2) == ARG and call(out=None) == ARG
    assert call(sm=float("inf")) == ARG
    assert call(sm=0.0) == ARG and call(sm=-0.1) == ARG  # masked scores are scaled
    assert call(max_pages=1 << 24) == UNS


def test_prefill_refuses_a_scale_that_is_flushed_to_zero():
    def call(sm):
        return hd.lib().hpc_prefill_attn_win(FAKE, FAKE, FAKE, 100, FAKE, 8, FAKE, 0, 8, 2, 128,
                                             300, 128, 4, sm, FAKE, None, None)

    assert call(2.0 ** -127) == E.HPC_ERR_ARG and call(2.0 ** -126) == E.HPC_OK


def test_write_refusals():
    P = E.hpc_rope_norm_params

    def call(qkv=FAKE, stride=1280, N=4, Hq=8, Hkv=1, D=128, B=4, kvs=FAKE, qout=FAKE, k=FAKE,
             params="default", req=None, max_pages=16, pages=10):
        p = P(1e-6, 1e6, 0, 1, None) if params == "default" else params
        return hd.lib().hpc_rope_norm_block(
            qkv, stride, FAKE, FAKE, FAKE, req, N, Hq, Hkv, D, FAKE, max_pages, B, k, FAKE, kvs,
            pages, qout, None, None, None if p is None else ctypes.byref(p), None)

    ARG, UNS = E.HPC_ERR_ARG, E.HPC_ERR_UNSUPPORTED
    assert call(N=0) == E.HPC_OK
    assert call(N=-1) == ARG and call(pages=0) == ARG
    assert call(D=64) == UNS and call(Hq=12, Hkv=8) == UNS
    assert call(stride=1272) == ARG and call(stride=1284) == ARG
    assert call(qkv=FAKE + 8) == ARG and call(kvs=FAKE + 4) == ARG and call(k=FAKE + 8) == ARG
    assert call(kvs=None) == ARG and call(qout=None) == ARG and call(qkv=None) == ARG
    assert call(N=5) == ARG  # token t is request t: needs N <= B
    assert call(params=None) == ARG
    for bad in (P(-1.0, 1e6, 0, 1, None), P(1e-6, 0.0, 0, 1, None), P(1e-6, 1e6, 2, 1, None),
                P(1e-6, 1e6, 0, 2, None), P(1e-6, 1e6, 0, 1, FAKE + 8)):
        assert call(params=bad) == ARG
    assert call(max_pages=(1 << 18) + 1) == UNS


def test_read_refusals():
    def call(k=FAKE, kvs=FAKE, pages=10, B=2, Hkv=1, D=128, ko=FAKE, out_pages=10, mp=8, omp=8,
             sl=FAKE):
        return hd.lib().hpc_kv_read_block(k, FAKE, kvs, pages, FAKE, mp, None, sl, B, Hkv, D, ko,
                                          FAKE, out_pages, FAKE, omp, None, None)

    ARG, UNS = E.HPC_ERR_ARG, E.HPC_ERR_UNSUPPORTED
    assert call(B=0) == E.HPC_OK
    assert call(B=-1) == ARG and call(Hkv=0) == ARG and call(pages=0) == ARG
    assert call(out_pages=0) == ARG and call(mp=0) == ARG and call(omp=0) == ARG
    assert call(D=64) == UNS and call(B=20000) == UNS
    assert call(mp=1 << 24, omp=1 << 24) == UNS
    assert call(k=None) == ARG and call(kvs=None) == ARG and call(sl=None) == ARG
    assert call(k=FAKE + 8) == ARG and call(ko=FAKE + 16) == ARG and call(kvs=FAKE + 4) == ARG


# ---------------------------------------------------------------- binding
@pytest.mark.skipif(torch.cuda.is_available(), reason="CPU tensors stand in for device ones")
def test_the_extension_looks_at_tensors():
    from load_balanced_paged_assign_gb300._tensors import dense
    f32, i32, bf16 = torch.float32, torch.int32, torch.bfloat16
    x, n = torch.zeros((3, 4)), torch.zeros(0, dtype=i32)
    s = torch.zeros((), dtype=bf16)
    assert dense(-1, (f32, i32, f32, bf16), x, n, None, s) == (
        (x.data_ptr(), n.data_ptr(), None, s.data_ptr()), ((3, 4), (0,), None, ()), (12, 0, None, 1))
    assert dense(-1, (f32, f32), x[1:], x[:, 1:]) == 1  # rows are dense, columns are not
    assert dense(-1, (f32, f32), x.T, x) == 0
    assert dense(-1, (i32,), x) == 0 and dense(0, (f32,), x) == 0
    assert dense(-1, (f32, f32), x, x.to("meta")) == 1
    assert dense(-1, (f32,), [1.0]) == 0 and dense(-1, ("f32",), x) == 0
    assert dense(-1, ()) == ((), (), ())
    for bad in ((-1, (f32,)), (-1, [f32], x), ("a", (f32,), x), (-1,)):
        with pytest.raises(TypeError):
            dense(*bad)
    for _ in range(1000):  # nothing it returns is kept or dropped once too often
        dense(-1, (f32, i32, f32), x, n, None)
        dense(-1, (f32, i32), x, x)


def test_binding_refuses_what_is_no_dense_array_of_its_type():
    bf16, e4m3 = torch.bfloat16, torch.float8_e4m3fn
    cache = torch.zeros((3, 64, 2, 128), dtype=bf16)
    c8 = torch.zeros((3, 64, 2, 128), dtype=e4m3)
    scale = torch.ones((3, 2, 2, 4))
    q = torch.zeros((2, 1, 4, 128), dtype=bf16)
    bt, sl = torch.zeros((2, 2), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    out = torch.zeros_like(q)
    po, pl = torch.zeros((9, 2, 128)), torch.zeros((9, 2))

    class Map:
        cap_desc, c = 9, E.hpc_task_map()

    def attn(q=q, k=cache, v=cache, kvs=None, bt=bt, out=out, po=po, done=None, Hkv=2):
        E.hpc_decode_attn_win(q, None, k, v, 1.0, 1.0, kvs, bt, sl, 4, Hkv, 1, 8, 0, 0.1, Map, po,
                              pl, out, done)

    for kw in (dict(k=cache.transpose(1, 2)), dict(k=cache.float()), dict(v=c8),
               dict(q=q.float()), dict(q=q[:1]), dict(k=cache[:, :, :1].contiguous()),
               dict(bt=bt.long()), dict(bt=bt[:1]), dict(kvs=scale),
               dict(k=c8, v=c8, q=q.to(e4m3), kvs=scale[:2]), dict(po=po[:3]), dict(out=out[:1]),
               dict(done=torch.zeros(1, dtype=torch.int32)), dict(Hkv=4)):
        with pytest.raises(ValueError):
            attn(**kw)
    with pytest.raises(ValueError):
        E.hpc_decode_plan_win(sl.long(), 2, 2, 8, 2, Map, window=3)
    for kw in (dict(q=q.float()), dict(q=q[:1]), dict(out=out[:1]), dict(bt=bt[:1]),
               dict(k=cache.transpose(1, 2))):
        a = dict(dict(q=q, k=cache, bt=bt, out=out), **kw)
        with pytest.raises(ValueError):
            E.hpc_prefill_attn_win(a["q"], a["k"], cache, a["bt"], sl, 4, 2, 1, 8, 0, 0.1, a["out"])
    pos = torch.zeros(3, dtype=torch.int32)
    w = torch.ones(128, dtype=bf16)
    qkv = torch.zeros((3, 8 * 128), dtype=bf16)
    qo = torch.zeros((3, 4, 128), dtype=bf16)
    for kw in (dict(qkv=qkv.float()), dict(qkv=qkv[:, ::2]), dict(qkv=qkv[:2]),
               dict(qkv=qkv[:, :900]), dict(w=w[:64]), dict(scale=scale[:, :1].contiguous()),
               dict(qo=qo[:2]), dict(qo=qo.to(e4m3)), dict(req=pos[:2]), dict(k=cache),
               dict(freq=torch.zeros(64))):
        a = dict(dict(qkv=qkv, w=w, scale=scale, qo=qo, req=pos, k=c8, freq=None), **kw)
        with pytest.raises(ValueError):
            E.hpc_rope_norm_block(a["qkv"], a["w"], w, pos, a["req"], 4, 2, bt, a["k"], c8,
                                  a["scale"], a["qo"], freq=a["freq"])
    for kw in (dict(ko=c8), dict(ko=cache.transpose(0, 1)), dict(st=pos), dict(obt=bt[:1]),
               dict(scale=scale.double())):
        a = dict(dict(ko=cache, st=None, obt=bt, scale=scale), **kw)
        with pytest.raises(ValueError):
            E.hpc_kv_read_block(c8, c8, a["scale"], bt, a["st"], sl, 2, a["ko"], cache, a["obt"])
