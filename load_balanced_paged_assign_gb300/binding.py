"""Python binding of the C ABI in include/hpc_decode.h (ctypes, argument marshalling only).

Every function here has the name of the C entry point it forwards to and does
nothing but turn torch tensors into pointers and sizes, call the library and
raise on a non-zero status.  All compute happens in libhpcdecode.so; there is
no fallback path: if the library is missing, every call raises.

A call is queued on `stream` (None: the current one) and runs behind what is queued
there, not behind other streams: tensors that are filled on another stream, or whose
memory the allocator took from work on another one, have to be waited for first, and
all of a call's tensors have to live until it has run.  The workspaces, task maps and
pools of this module are ready for any stream when their constructors return.
"""

from __future__ import annotations

import ctypes
import os

import torch

from . import _build

HPC_OK, HPC_ERR_ARG, HPC_ERR_UNSUPPORTED, HPC_ERR_WORKSPACE, HPC_ERR_CUDA = 0, -1, -2, -3, -4
HPC_KV_BF16, HPC_KV_FP8_E4M3, HPC_KV_E4M3_BLOCK = 0, 1, 2
HPC_FLAG_BAD_SEQLEN, HPC_FLAG_DESC_OVERFLOW, HPC_FLAG_BAD_PAGE, HPC_FLAG_TIMEOUT = 1, 2, 4, 8
HPC_FLAG_NO_PAGES = 16
HEAD_DIM, PAGE_SIZE, MAX_GROUP, MAX_QUERY_ROWS = 128, 64, 16, 16
SCALE_BLOCK = 16
HPC_ROPE_HALVES, HPC_ROPE_INTERLEAVED = 0, 1

# Every symbol the header declares; the CPU tests check the library exports them all.
EXPORTS = (
    "hpc_decode_version", "hpc_status_string", "hpc_decode_num_ctas", "hpc_decode_desc_capacity",
    "hpc_decode_static_capacity", "hpc_decode_plan", "hpc_decode_plan_static", "hpc_decode_attn",
    "hpc_decode_attn_combine", "hpc_decode_combine", "hpc_decode_step", "hpc_decode_step_host", "hpc_decode_read_meta",
    "hpc_decode_step_noalloc", "hpc_rope_norm", "hpc_rope_frequencies", "hpc_decode_attn_mq",
    "hpc_decode_attn_combine_mq", "hpc_decode_combine_mq", "hpc_decode_step_mq",
    "hpc_selftest_wait_timeout", "hpc_router_split", "hpc_router_workspace_bytes", "hpc_router_plan",
    "hpc_router_gemm", "hpc_prefill_attn",
    "hpc_decode_packed_layout", "hpc_decode_step_host_packed",
    "hpc_decode_plan_win", "hpc_decode_attn_win", "hpc_decode_step_win", "hpc_prefill_attn_win",
    "hpc_rope_norm_block", "hpc_kv_read_block",
    "hpc_kv_free", "hpc_kv_extend", "hpc_kv_fork", "hpc_kv_compact", "hpc_kv_copy_pages",
    "hpc_decode_shared_capacity", "hpc_decode_plan_shared", "hpc_decode_attn_shared",
    "hpc_decode_step_shared",
)


class HpcError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


class hpc_task_map(ctypes.Structure):
    _fields_ = [
        ("desc", ctypes.c_void_p), ("bin_ptr", ctypes.c_void_p),
        ("chunk_count", ctypes.c_void_p), ("chunk_off", ctypes.c_void_p),
        ("meta", ctypes.c_void_p),
        ("cap_desc", ctypes.c_int32), ("cap_bins", ctypes.c_int32), ("cap_units", ctypes.c_int32),
        ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
        ("persistent", ctypes.c_int32), ("min_tiles", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("q_len", ctypes.c_int32), ("window", ctypes.c_int32),
        ("sinks", ctypes.c_int32),
    ]


class hpc_rope_norm_params(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("rope_base", ctypes.c_float),
                ("rope_layout", ctypes.c_int32), ("norm_first", ctypes.c_int32),
                ("freq", ctypes.c_void_p)]


class hpc_page_pool(ctypes.Structure):
    _fields_ = [("refs", ctypes.c_void_p), ("free_list", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("marks", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


class hpc_shared_map(ctypes.Structure):
    _fields_ = [("tail", hpc_task_map), ("head", ctypes.c_void_p), ("head_o", ctypes.c_void_p),
                ("head_lse", ctypes.c_void_p), ("cap_head", ctypes.c_int64),
                ("cap_slots", ctypes.c_int64), ("Hq", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


_LIB = None


def library_path() -> str:
    """The in-tree library, or the file named by HPC_DECODE_LIB (another build
    of the same sources, e.g. with a different pipeline shape)."""
    return os.environ.get("HPC_DECODE_LIB") or _build.LIB_PATH


def lib():
    """The loaded libhpcdecode.so; raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(path)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    tm, pool = ctypes.POINTER(hpc_task_map), ctypes.POINTER(hpc_page_pool)
    sm = ctypes.POINTER(hpc_shared_map)
    sig = {
        "hpc_decode_version": (ctypes.c_char_p, []),
        "hpc_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hpc_decode_num_ctas": (i32, [i32, ctypes.c_int]),
        "hpc_decode_desc_capacity": (i64, [i32, i32, i32]),
        "hpc_decode_static_capacity": (i64, [i32, i32, i32]),
        "hpc_decode_plan": (ctypes.c_int, [vp, i32, i32, i32, i32, i32, tm, vp]),
        "hpc_decode_plan_static": (ctypes.c_int, [vp, i32, i32, i32, i32, tm, vp]),
        "hpc_decode_attn": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int, vp, i32,
                                           vp, i32, i32, i32, i32, f32, tm, vp, vp, vp]),
        "hpc_decode_attn_combine": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int,
                                                   vp, i32, vp, i32, i32, i32, i32, f32, tm, vp,
                                                   vp, vp, vp, vp]),
        "hpc_decode_combine": (ctypes.c_int, [vp, vp, tm, i32, i32, i32, i32, vp, vp]),
        "hpc_decode_step": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int, vp, i32,
                                           vp, i32, i32, i32, i32, f32, i32, i32, i32, tm, vp,
                                           vp, vp, vp, vp]),
        "hpc_decode_step_host": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                i32, f32, f32, ctypes.c_int, i32, i32, i32, i32,
                                                i32, f32, i32, i32, i32, tm, vp, vp, vp, vp]),
        "hpc_decode_read_meta": (ctypes.c_int, [tm, ctypes.POINTER(ctypes.c_int32), vp]),
        "hpc_decode_step_noalloc": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int,
                                                   vp, i32, vp, i32, i32, i32, i32, f32, i32, i32,
                                                   vp, vp, vp]),
        "hpc_rope_frequencies": (ctypes.c_int, [f32, vp, vp]),
        "hpc_router_split": (ctypes.c_int, [vp, i32, i32, vp, vp, vp]),
        "hpc_router_workspace_bytes": (i64, [i32, i32, i32]),
        "hpc_router_plan": (ctypes.c_int, [i32, i32, i32, vp]),
        "hpc_selftest_wait_timeout": (ctypes.c_int, [vp, i32, vp]),
        "hpc_router_gemm": (ctypes.c_int, [vp, vp, vp, i32, i32, i32, vp, vp, i64, vp, vp]),
        "hpc_prefill_attn": (ctypes.c_int, [vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32,
                                            i32, f32, vp, vp, vp]),
        "hpc_decode_packed_layout": (i64, [i32, i32, i32, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_int64)]),
        "hpc_decode_step_host_packed": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, i32, f32, f32,
                                                       ctypes.c_int, i32, i32, i32, i32, i32, f32,
                                                       i32, i32, i32, tm, vp, vp, vp, vp]),
        "hpc_decode_attn_mq": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int, vp,
                                              i32, vp, i32, i32, i32, i32, i32, f32, tm, vp, vp,
                                              vp]),
        "hpc_decode_attn_combine_mq": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int,
                                                      vp, i32, vp, i32, i32, i32, i32, i32, f32,
                                                      tm, vp, vp, vp, vp, vp]),
        "hpc_decode_combine_mq": (ctypes.c_int, [vp, vp, tm, i32, i32, i32, i32, i32, vp, vp]),
        "hpc_decode_step_mq": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, ctypes.c_int, vp,
                                              i32, vp, i32, i32, i32, i32, i32, f32, i32, i32,
                                              i32, tm, vp, vp, vp, vp, vp]),
        "hpc_rope_norm": (ctypes.c_int, [vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp, i32,
                                         i32, vp, vp, i32, ctypes.c_int, f32, f32, vp, vp, vp,
                                         ctypes.POINTER(hpc_rope_norm_params), vp]),
        "hpc_decode_plan_win": (ctypes.c_int, [vp, i32, i32, i32, i32, i32, ctypes.c_int, i32,
                                               i32, i32, tm, vp]),
        "hpc_decode_attn_win": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, vp, ctypes.c_int,
                                               vp, i32, vp, i32, i32, i32, i32, i32, i32, i32,
                                               f32, tm, vp, vp, vp, vp, vp]),
        "hpc_decode_step_win": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, vp, ctypes.c_int,
                                               vp, i32, vp, i32, i32, i32, i32, i32, i32, i32,
                                               f32, i32, i32, tm, vp, vp, vp, vp, vp]),
        "hpc_prefill_attn_win": (ctypes.c_int, [vp, vp, vp, i32, vp, i32, vp, i32, i32, i32, i32,
                                                i32, i32, i32, f32, vp, vp, vp]),
        "hpc_rope_norm_block": (ctypes.c_int, [vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp,
                                               i32, i32, vp, vp, vp, i32, vp, vp, vp,
                                               ctypes.POINTER(hpc_rope_norm_params), vp]),
        "hpc_kv_read_block": (ctypes.c_int, [vp, vp, vp, i32, vp, i32, vp, vp, i32, i32, i32, vp,
                                             vp, i32, vp, i32, vp, vp]),
        "hpc_decode_shared_capacity": (ctypes.c_int, [i32, i32, i32, i32, i32, i32,
                                                      ctypes.POINTER(i64)]),
        "hpc_decode_plan_shared": (ctypes.c_int, [vp, i32, i32, i32, i32, vp, vp, i32, i32, i32,
                                                  ctypes.c_int, i32, sm, vp]),
        "hpc_decode_attn_shared": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, vp, ctypes.c_int,
                                                  vp, i32, vp, i32, i32, i32, i32, i32, f32, sm,
                                                  vp, vp, vp, vp]),
        "hpc_decode_step_shared": (ctypes.c_int, [vp, vp, vp, vp, i32, f32, f32, vp, ctypes.c_int,
                                                  vp, i32, vp, vp, vp, i32, i32, i32, i32, i32,
                                                  i32, f32, i32, i32, sm, vp, vp, vp, vp]),
        "hpc_kv_free": (ctypes.c_int, [pool, vp, i32, i32, vp, vp, i32, vp]),
        "hpc_kv_extend": (ctypes.c_int, [pool, vp, i32, i32, vp, vp, i32, vp]),
        "hpc_kv_fork": (ctypes.c_int, [pool, vp, i32, i32, vp, vp, vp, i32, vp, i32, vp]),
        "hpc_kv_compact": (ctypes.c_int, [pool, vp, i32, i32, vp, i32, vp, pool, vp]),
        "hpc_kv_copy_pages": (ctypes.c_int, [vp, i32, vp, vp, vp, ctypes.c_int, i32, i32, i32, vp,
                                             vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    _LIB = L
    return L


def status_string(status: int) -> str:
    try:
        return lib().hpc_status_string(int(status)).decode()
    except RuntimeError:
        return "unknown"


def _check(fn: str, status: int):
    if status != HPC_OK:
        raise HpcError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def kv_dtype_of(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return HPC_KV_BF16
    if t.dtype == torch.float8_e4m3fn:
        return HPC_KV_FP8_E4M3
    raise TypeError(f"unsupported KV cache dtype {t.dtype}")


_DENSE = None  # _tensors.dense, once a call has needed it
_BF16, _E4M3, _F32, _F64, _I32 = (torch.bfloat16, torch.float8_e4m3fn, torch.float32,
                                  torch.float64, torch.int32)


def _load_dense():
    global _DENSE
    how = "(python -c 'import __graft_entry__ as g; g.build()')"
    built = _build.extension_built_for()
    if built is not None and built != _build.extension_target():
        raise RuntimeError("the extension module _tensors was built for another PyTorch or Python "
                           f"({built or 'unknown'}): build it again {how}")
    try:
        from . import _tensors
    except ImportError as e:
        why = "is missing: build it first" if built is None else \
            f"cannot be loaded ({e}): build it again"
        raise RuntimeError(f"the extension module _tensors {why} {how}") from e
    _DENSE = _tensors.dense
    return _DENSE


def _arrays(fn: str, dev: int, names: str, types: tuple, *tensors) -> tuple:
    """The tensors' (addresses, shapes, element counts), None for None; raises for the first
    that is no row-major array of its type on the device `dev`, as the library takes its
    pointers to be."""
    got = (_DENSE or _load_dense())(dev, types, *tensors)
    if type(got) is int:
        t, name, dtype = tensors[got], names.split()[got], types[got]
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{fn}: {name} is a {type(t).__name__}, not a tensor")
        why = f"{t.dtype}, not {dtype}" if t.dtype is not dtype else \
            "not contiguous" if not t.is_contiguous() else \
            f"on {t.device}, not on the current device"
        raise ValueError(f"{fn}: {name} is {why}")
    return got


def _shape(fn: str, name: str, shape: tuple, want: tuple):
    if shape != want:
        raise ValueError(f"{fn}: {name} is {shape}, not {want}")


def _table(fn: str, name: str, shape: tuple, B: int):
    if len(shape) != 2 or shape[0] < B:
        raise ValueError(f"{fn}: {name} has not a row for each of the {B} requests")


_HAS_CUDA = None


def _current_device() -> int:
    """The current CUDA device, or -1 (the device number of CPU tensors) without one."""
    global _HAS_CUDA
    if _HAS_CUDA is None:
        _HAS_CUDA = torch.cuda.is_available()
    return torch._C._cuda_getDevice() if _HAS_CUDA else -1


def _raw_stream(dev: int, stream):
    """The stream's handle; None: the current stream of `dev`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ready(dev: torch.device):
    """Waits for the current stream, on which new tensors are filled, and by which alone the
    allocator orders their memory's earlier use: then any stream may use them.  Part of a
    graph while one is captured (they belong to that graph)."""
    if dev.type == "cuda" and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(dev).synchronize()


class TaskMap:
    """Caller-owned device buffers of one task map and the C struct describing them.  It is
    ready for calls on any stream when it is made, as workspaces and pools are; like them it
    has to outlive the work that uses it."""

    def __init__(self, B: int, Hkv: int, cap_desc: int, cap_bins: int, device="cuda"):
        dev = torch.device(device)
        self.desc = torch.zeros((max(cap_desc, 1), 4), dtype=torch.int32, device=dev)
        self.bin_ptr = torch.zeros(max(cap_bins, 1), dtype=torch.int32, device=dev)
        units = max(B * Hkv, 1)
        self.chunk_count = torch.zeros(units, dtype=torch.int32, device=dev)
        self.chunk_off = torch.zeros(units, dtype=torch.int32, device=dev)
        self.meta = torch.zeros(8, dtype=torch.int32, device=dev)
        self.c = hpc_task_map(_ptr(self.desc), _ptr(self.bin_ptr), _ptr(self.chunk_count),
                              _ptr(self.chunk_off), _ptr(self.meta), cap_desc, cap_bins, units)
        _ready(dev)

    @classmethod
    def dynamic(cls, B: int, Hkv: int, num_ctas: int, device="cuda"):
        return cls(B, Hkv, int(lib().hpc_decode_desc_capacity(B, Hkv, num_ctas)), num_ctas + 1,
                   device)

    @classmethod
    def static(cls, B: int, Hkv: int, num_splits: int, device="cuda"):
        n = int(lib().hpc_decode_static_capacity(B, Hkv, num_splits))
        return cls(B, Hkv, n, n + 1, device)

    @property
    def cap_desc(self) -> int:
        return int(self.c.cap_desc)

    @property
    def num_ctas(self) -> int:
        return int(self.c.num_ctas)

    def to_host(self) -> dict:
        """The map as host lists (synchronises the current stream)."""
        meta = self.meta.tolist()
        n = int(meta[2])
        units = int(self.c.B) * int(self.c.Hkv) // (2 if self.c.persistent & 2 else 1)  # pairs
        return dict(total_tiles=meta[0], budget=meta[1], num_desc=n, flags=meta[3],
                    desc=[tuple(d) for d in self.desc[:n].tolist()],
                    bin_ptr=self.bin_ptr[:self.num_ctas + 1].tolist(),
                    chunk_count=self.chunk_count[:units].tolist(),
                    chunk_off=self.chunk_off[:units].tolist())


def hpc_decode_version() -> str:
    return lib().hpc_decode_version().decode()


def hpc_decode_num_ctas(device: int = 0, kv_dtype: int = HPC_KV_BF16) -> int:
    n = int(lib().hpc_decode_num_ctas(int(device), int(kv_dtype)))
    if n < 0:
        raise HpcError("hpc_decode_num_ctas", n)
    return n


def hpc_decode_desc_capacity(B: int, Hkv: int, num_ctas: int) -> int:
    return int(lib().hpc_decode_desc_capacity(B, Hkv, num_ctas))


def hpc_decode_static_capacity(B: int, Hkv: int, num_splits: int) -> int:
    return int(lib().hpc_decode_static_capacity(B, Hkv, num_splits))


def hpc_decode_plan(seqlens, Hkv, max_pages_per_req, num_ctas, min_tiles_per_cta, tmap: TaskMap,
                    stream=None):
    B = int(seqlens.numel())
    _check("hpc_decode_plan", lib().hpc_decode_plan(
        _ptr(seqlens), B, int(Hkv), int(max_pages_per_req), int(num_ctas),
        int(min_tiles_per_cta), ctypes.byref(tmap.c), _stream(stream)))


def hpc_decode_plan_static(seqlens, Hkv, max_pages_per_req, num_splits, tmap: TaskMap,
                           stream=None):
    B = int(seqlens.numel())
    _check("hpc_decode_plan_static", lib().hpc_decode_plan_static(
        _ptr(seqlens), B, int(Hkv), int(max_pages_per_req), int(num_splits),
        ctypes.byref(tmap.c), _stream(stream)))


def hpc_decode_attn(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, Hq, Hkv,
                    sm_scale, tmap: TaskMap, part_o, part_lse, stream=None):
    _check("hpc_decode_attn", lib().hpc_decode_attn(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, float(sm_scale), ctypes.byref(tmap.c), _ptr(part_o), _ptr(part_lse),
        _stream(stream)))


def hpc_decode_attn_combine(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, seqlens,
                            Hq, Hkv, sm_scale, tmap: TaskMap, part_o, part_lse, unit_done, out,
                            stream=None):
    _check("hpc_decode_attn_combine", lib().hpc_decode_attn_combine(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, float(sm_scale), ctypes.byref(tmap.c), _ptr(part_o), _ptr(part_lse),
        _ptr(unit_done), _ptr(out), _stream(stream)))


def hpc_decode_combine(part_o, part_lse, tmap: TaskMap, B, Hq, Hkv, out, stream=None):
    _check("hpc_decode_combine", lib().hpc_decode_combine(
        _ptr(part_o), _ptr(part_lse), ctypes.byref(tmap.c), int(B), int(Hq), int(Hkv), HEAD_DIM,
        _ptr(out), _stream(stream)))


def hpc_decode_step(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, Hq,
                    Hkv, sm_scale, num_ctas, min_tiles_per_cta, num_splits, tmap: TaskMap, part_o,
                    part_lse, out, unit_done=None, stream=None):
    """unit_done given: fused attention + combine; None: separate combine kernel."""
    _check("hpc_decode_step", lib().hpc_decode_step(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, float(sm_scale), int(num_ctas), int(min_tiles_per_cta), int(num_splits),
        ctypes.byref(tmap.c), _ptr(part_o), _ptr(part_lse), _ptr(unit_done), _ptr(out),
        _stream(stream)))


def hpc_decode_attn_mq(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, Hq,
                       Hkv, q_len, sm_scale, tmap: TaskMap, part_o, part_lse, stream=None):
    """Multi-query attention: q [B, q_len, Hq, 128]; partials [cap, q_len * G, ...]."""
    _check("hpc_decode_attn_mq", lib().hpc_decode_attn_mq(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, int(q_len), float(sm_scale), ctypes.byref(tmap.c), _ptr(part_o),
        _ptr(part_lse), _stream(stream)))


def hpc_decode_attn_combine_mq(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table,
                               seqlens, Hq, Hkv, q_len, sm_scale, tmap: TaskMap, part_o, part_lse,
                               unit_done, out, stream=None):
    _check("hpc_decode_attn_combine_mq", lib().hpc_decode_attn_combine_mq(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, int(q_len), float(sm_scale), ctypes.byref(tmap.c), _ptr(part_o),
        _ptr(part_lse), _ptr(unit_done), _ptr(out), _stream(stream)))


def hpc_decode_combine_mq(part_o, part_lse, tmap: TaskMap, B, Hq, Hkv, q_len, out, stream=None):
    _check("hpc_decode_combine_mq", lib().hpc_decode_combine_mq(
        _ptr(part_o), _ptr(part_lse), ctypes.byref(tmap.c), int(B), int(Hq), int(Hkv), HEAD_DIM,
        int(q_len), _ptr(out), _stream(stream)))


def hpc_decode_step_mq(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, seqlens, Hq,
                       Hkv, q_len, sm_scale, num_ctas, min_tiles_per_cta, num_splits,
                       tmap: TaskMap, part_o, part_lse, out, unit_done=None, stream=None):
    """hpc_decode_step with q_len query tokens per request (causal among them)."""
    _check("hpc_decode_step_mq", lib().hpc_decode_step_mq(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, int(q_len), float(sm_scale), int(num_ctas), int(min_tiles_per_cta),
        int(num_splits), ctypes.byref(tmap.c), _ptr(part_o), _ptr(part_lse), _ptr(unit_done),
        _ptr(out), _stream(stream)))


def hpc_router_split(w, w_hi, w_lo, stream=None):
    """Split fp32 router weights [N, K] into BF16 W_high / W_low [N, K]."""
    N, K = w.shape
    _check("hpc_router_split", lib().hpc_router_split(_ptr(w), int(N), int(K), _ptr(w_hi),
                                                        _ptr(w_lo), _stream(stream)))


def hpc_router_workspace_bytes(M, N, K) -> int:
    return int(lib().hpc_router_workspace_bytes(int(M), int(N), int(K)))


def hpc_selftest_wait_timeout(flags, limit_us, stream=None):
    """One CTA waits on a barrier nothing completes for limit_us, then raises
    HPC_FLAG_TIMEOUT in flags (device int32) and returns."""
    _check("hpc_selftest_wait_timeout",
           lib().hpc_selftest_wait_timeout(_ptr(flags), int(limit_us), _stream(stream)))


def hpc_router_plan(M, N, K) -> dict:
    """The launch hpc_router_gemm makes for this shape on the current device."""
    plan = (ctypes.c_int32 * 4)()
    _check("hpc_router_plan", lib().hpc_router_plan(int(M), int(N), int(K), plan))
    return {"tensor_cores": bool(plan[0]), "bn": int(plan[1]), "splits": int(plan[2]),
            "ctas": int(plan[3])}


def hpc_router_gemm(x, w_hi, w_lo, out, workspace=None, flags=None, stream=None):
    """Router scores out [M, N] fp32 = X W_high^T + (X W_low^T) / 256."""
    M, K = x.shape
    N = w_hi.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("hpc_router_gemm", lib().hpc_router_gemm(
        _ptr(x), _ptr(w_hi), _ptr(w_lo), int(M), int(N), int(K), _ptr(out), _ptr(workspace),
        int(ws_bytes), _ptr(flags), _stream(stream)))


def hpc_prefill_attn(q, k_cache, v_cache, block_table, seqlens, Hq, Hkv, q_len, sm_scale, out,
                     flags=None, stream=None):
    """Extend / prefill attention: q and out [B, q_len, Hq, 128] bf16, causal
    over each request's last q_len live tokens."""
    _check("hpc_prefill_attn", lib().hpc_prefill_attn(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, int(q_len), float(sm_scale), _ptr(out), _ptr(flags), _stream(stream)))


def hpc_decode_step_host(h_q, h_q_scale, h_seqlens, h_block_table, h_out, d_q, d_q_scale,
                         d_seqlens, d_block_table, d_out, k_cache, v_cache, k_scale, v_scale, Hq,
                         Hkv, sm_scale, num_ctas, min_tiles_per_cta, num_splits, tmap: TaskMap,
                         part_o, part_lse, unit_done=None, stream=None):
    _check("hpc_decode_step_host", lib().hpc_decode_step_host(
        _ptr(h_q), _ptr(h_q_scale), _ptr(h_seqlens), _ptr(h_block_table), _ptr(h_out), _ptr(d_q),
        _ptr(d_q_scale), _ptr(d_seqlens), _ptr(d_block_table), _ptr(d_out), _ptr(k_cache),
        _ptr(v_cache), int(k_cache.shape[0]), float(k_scale), float(v_scale),
        kv_dtype_of(k_cache), int(h_block_table.shape[1]), int(h_seqlens.numel()), int(Hq),
        int(Hkv), HEAD_DIM, float(sm_scale), int(num_ctas), int(min_tiles_per_cta),
        int(num_splits), ctypes.byref(tmap.c), _ptr(part_o), _ptr(part_lse), _ptr(unit_done),
        _stream(stream)))


def hpc_decode_packed_layout(B, Hq, max_pages, kv_dtype=HPC_KV_BF16):
    """(total bytes, [q, q_scale or -1, seqlens, block_table] byte offsets) of the
    packed per-step input."""
    off = (ctypes.c_int64 * 4)()
    total = int(lib().hpc_decode_packed_layout(int(B), int(Hq), int(max_pages), int(kv_dtype),
                                                 off))
    if total < 0:
        raise HpcError("hpc_decode_packed_layout", HPC_ERR_ARG)
    return total, list(off)


def hpc_decode_step_host_packed(h_in, d_in, h_out, d_out, k_cache, v_cache, k_scale, v_scale, B,
                                Hq, Hkv, max_pages, sm_scale, num_ctas, min_tiles_per_cta,
                                num_splits, tmap: TaskMap, part_o, part_lse, unit_done=None,
                                stream=None):
    """One decode step from one packed pinned host buffer (see hpc_decode_packed_layout)."""
    _check("hpc_decode_step_host_packed", lib().hpc_decode_step_host_packed(
        _ptr(h_in), _ptr(d_in), _ptr(h_out), _ptr(d_out), _ptr(k_cache), _ptr(v_cache),
        int(k_cache.shape[0]), float(k_scale), float(v_scale), kv_dtype_of(k_cache),
        int(max_pages), int(B), int(Hq), int(Hkv), HEAD_DIM, float(sm_scale), int(num_ctas),
        int(min_tiles_per_cta), int(num_splits), ctypes.byref(tmap.c), _ptr(part_o),
        _ptr(part_lse), _ptr(unit_done), _stream(stream)))


def hpc_decode_read_meta(tmap: TaskMap, stream=None) -> list:
    host = (ctypes.c_int32 * 4)()
    _check("hpc_decode_read_meta", lib().hpc_decode_read_meta(ctypes.byref(tmap.c), host,
                                                              _stream(stream)))
    return list(host)


def hpc_decode_step_noalloc(q, q_scale, k_cache, v_cache, k_scale, v_scale, block_table, seqlens,
                            Hq, Hkv, sm_scale, num_ctas, min_tiles_per_cta, out, meta_out=None,
                            stream=None):
    """Whole step with the library's built-in scratch; see the C header."""
    _check("hpc_decode_step_noalloc", lib().hpc_decode_step_noalloc(
        _ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]),
        float(k_scale), float(v_scale), kv_dtype_of(k_cache), _ptr(block_table),
        int(block_table.shape[1]), _ptr(seqlens), int(seqlens.numel()), int(Hq), int(Hkv),
        HEAD_DIM, float(sm_scale), int(num_ctas), int(min_tiles_per_cta), _ptr(out),
        _ptr(meta_out), _stream(stream)))


def hpc_rope_frequencies(rope_base, freq, stream=None):
    """The fp64 RoPE frequency table [64] for rope_base, written into `freq`."""
    _check("hpc_rope_frequencies",
           lib().hpc_rope_frequencies(float(rope_base), _ptr(freq), _stream(stream)))


def hpc_rope_norm(qkv, q_norm_w, k_norm_w, positions, token_req, Hq, Hkv, block_table, k_cache,
                  v_cache, k_scale, v_scale, q_out, q_scale_out=None, flags=None, *, eps=1e-6,
                  rope_base=1e6, rope_layout=HPC_ROPE_HALVES, norm_first=True, freq=None,
                  stream=None):
    """Fused prologue: QK-Norm + RoPE of the new tokens' heads, K/V written into
    the paged cache, the query into q_out (and q_scale_out for FP8).  `freq`:
    the table from hpc_rope_frequencies(rope_base), or None."""
    params = hpc_rope_norm_params(float(eps), float(rope_base), int(rope_layout),
                                  1 if norm_first else 0,
                                  None if freq is None else freq.data_ptr())
    _check("hpc_rope_norm", lib().hpc_rope_norm(
        _ptr(qkv), int(qkv.stride(0)), _ptr(q_norm_w), _ptr(k_norm_w), _ptr(positions),
        _ptr(token_req), int(positions.numel()), int(Hq), int(Hkv), HEAD_DIM, _ptr(block_table),
        int(block_table.shape[1]), int(block_table.shape[0]), _ptr(k_cache), _ptr(v_cache),
        int(k_cache.shape[0]), kv_dtype_of(k_cache), float(k_scale), float(v_scale), _ptr(q_out),
        _ptr(q_scale_out), _ptr(flags), ctypes.byref(params), _stream(stream)))


def hpc_decode_plan_win(seqlens, Hkv, max_pages_per_req, num_ctas, min_tiles_per_cta,
                        tmap: TaskMap, *, kv_dtype=HPC_KV_BF16, q_len=1, window=0, sinks=0,
                        stream=None):
    """hpc_decode_plan for queries that see the last `window` tokens and the
    first `sinks` ones (window = 0: every token) of a kv_dtype cache."""
    dev = _current_device()
    (adr,), _, (B,) = _arrays("hpc_decode_plan_win", dev, "seqlens", (_I32,), seqlens)
    _check("hpc_decode_plan_win", lib().hpc_decode_plan_win(
        adr, B, int(Hkv), int(max_pages_per_req), int(num_ctas),
        int(min_tiles_per_cta), int(kv_dtype), int(q_len), int(window), int(sinks),
        ctypes.byref(tmap.c),
        _raw_stream(dev, stream)))


_WIN_NAMES = ("q k_cache v_cache q_scale kv_scale block_table seqlens part_o part_lse unit_done "
              "out")
_WIN_TYPES = [(t, t, t, _F32, _F32, _I32, _I32, _F32, _F32, _I32, _BF16) for t in (_BF16, _E4M3)]


def _win_args(fn, q, q_scale, k_cache, v_cache, kv_scale, block_table, seqlens, Hq, Hkv, q_len,
              part_o, part_lse, out, unit_done, cap_desc):
    """The checks of the windowed decode calls; returns (KV dtype, device, requests, pages,
    pages per request, addresses in the order of _WIN_NAMES)."""
    block, dev = kv_scale is not None, _current_device()
    e4m3 = block or k_cache.dtype is _E4M3
    adr, shape, count = _arrays(fn, dev, _WIN_NAMES, _WIN_TYPES[e4m3], q, k_cache, v_cache, q_scale,
                                kv_scale, block_table, seqlens, part_o, part_lse, unit_done, out)
    pages, table, B = shape[1][0] if shape[1] else 0, shape[5], count[6]
    rows, want = B * q_len * Hq, (pages, PAGE_SIZE, Hkv, HEAD_DIM)
    _shape(fn, "k_cache", shape[1], want)
    _shape(fn, "v_cache", shape[2], want)
    if block:
        _shape(fn, "kv_scale", shape[4], (pages, Hkv, 2, PAGE_SIZE // SCALE_BLOCK))
    _table(fn, "block_table", table, B)
    if count[0] != rows * HEAD_DIM or (out is not None and count[10] < rows * HEAD_DIM):
        raise ValueError(f"{fn}: q or out does not hold {B} x {q_len} x {Hq} rows")
    if q_scale is not None and count[3] != rows:
        raise ValueError(f"{fn}: q_scale does not hold {B} x {q_len} x {Hq} scales")
    # room in the split buffer and the counters for what the map may hold
    rows = cap_desc * q_len * (Hq // max(Hkv, 1))
    if count[7] < rows * HEAD_DIM or count[8] < rows:
        raise ValueError(f"{fn}: part_o or part_lse is smaller than the map's {cap_desc} "
                         f"descriptors need")
    if unit_done is not None and count[9] < B * Hkv:
        raise ValueError(f"{fn}: unit_done holds fewer than {B} x {Hkv} counters")
    kv = HPC_KV_E4M3_BLOCK if block else HPC_KV_FP8_E4M3 if e4m3 else HPC_KV_BF16
    return kv, dev, B, pages, table[1], adr


def hpc_decode_attn_win(q, q_scale, k_cache, v_cache, k_scale, v_scale, kv_scale, block_table,
                        seqlens, Hq, Hkv, q_len, window, sinks, sm_scale, tmap: TaskMap, part_o,
                        part_lse, out=None, unit_done=None, stream=None):
    """Attention over a window with sinks (window = 0: every token) on a map from
    hpc_decode_plan_win.  kv_scale: the block scales [num_pages, Hkv, 2, 4] of a
    block-scaled cache, else None.  out and unit_done given: combine fused in;
    both None: partials only."""
    fn = "hpc_decode_attn_win"
    Hq, Hkv, q_len = int(Hq), int(Hkv), int(q_len)
    kv, dev, B, pages, cols, (q_, k_, v_, qs_, sc_, bt_, sl_, po_, pl_, ud_, out_) = _win_args(
        fn, q, q_scale, k_cache, v_cache, kv_scale, block_table, seqlens, Hq, Hkv, q_len, part_o,
        part_lse, out, unit_done, tmap.cap_desc)
    status = lib().hpc_decode_attn_win(
        q_, qs_, k_, v_, pages, float(k_scale), float(v_scale), sc_, kv, bt_, cols, sl_, B, Hq,
        Hkv, HEAD_DIM, q_len, int(window), int(sinks),
        float(sm_scale), ctypes.byref(tmap.c), po_, pl_, ud_, out_,
        _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_decode_step_win(q, q_scale, k_cache, v_cache, k_scale, v_scale, kv_scale, block_table,
                        seqlens, Hq, Hkv, q_len, window, sinks, sm_scale, num_ctas,
                        min_tiles_per_cta, tmap: TaskMap, part_o, part_lse, out, unit_done=None,
                        stream=None):
    """hpc_decode_plan_win and hpc_decode_attn_win in one call (unit_done None:
    with the separate combine kernel)."""
    fn = "hpc_decode_step_win"
    Hq, Hkv, q_len = int(Hq), int(Hkv), int(q_len)
    kv, dev, B, pages, cols, (q_, k_, v_, qs_, sc_, bt_, sl_, po_, pl_, ud_, out_) = _win_args(
        fn, q, q_scale, k_cache, v_cache, kv_scale, block_table, seqlens, Hq, Hkv, q_len, part_o,
        part_lse, out, unit_done, tmap.cap_desc)
    status = lib().hpc_decode_step_win(
        q_, qs_, k_, v_, pages, float(k_scale), float(v_scale), sc_, kv, bt_, cols, sl_, B, Hq,
        Hkv, HEAD_DIM, q_len, int(window), int(sinks),
        float(sm_scale), int(num_ctas), int(min_tiles_per_cta), ctypes.byref(tmap.c), po_, pl_, ud_,
        out_, _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_prefill_attn_win(q, k_cache, v_cache, block_table, seqlens, Hq, Hkv, q_len, window, sinks,
                         sm_scale, out, flags=None, stream=None):
    """hpc_prefill_attn with a window and sinks (window = 0: plain causal)."""
    fn, dev = "hpc_prefill_attn_win", _current_device()
    Hq, Hkv, q_len = int(Hq), int(Hkv), int(q_len)
    (q_, k_, v_, out_, bt_, sl_, fl_), shape, count = _arrays(
        fn, dev, "q k_cache v_cache out block_table seqlens flags",
        (_BF16, _BF16, _BF16, _BF16, _I32, _I32, _I32), q, k_cache, v_cache, out, block_table,
        seqlens, flags)
    B, pages, table = count[5], shape[1][0] if shape[1] else 0, shape[4]
    want, n = (pages, PAGE_SIZE, Hkv, HEAD_DIM), B * q_len * Hq * HEAD_DIM
    _shape(fn, "k_cache", shape[1], want)
    _shape(fn, "v_cache", shape[2], want)
    _table(fn, "block_table", table, B)
    if count[0] != n or count[3] < n:
        raise ValueError(f"{fn}: q or out does not hold {B} x {q_len} x {Hq} rows")
    status = lib().hpc_prefill_attn_win(
        q_, k_, v_, pages, bt_, table[1], sl_, B, Hq, Hkv, HEAD_DIM, q_len,
        int(window), int(sinks), float(sm_scale), out_, fl_, _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


_WRITE_TYPES = [(_BF16, _BF16, _I32, _I32, _I32, _E4M3, _E4M3, _F32, q, _F32, _I32, _F64)
                for q in (_BF16, _E4M3)]  # BF16 queries, E4M3 queries


def hpc_rope_norm_block(qkv, q_norm_w, k_norm_w, positions, token_req, Hq, Hkv, block_table,
                        k_cache, v_cache, kv_scale, q_out, q_scale_out=None, flags=None, *,
                        eps=1e-6, rope_base=1e6, rope_layout=HPC_ROPE_HALVES, norm_first=True,
                        freq=None, stream=None):
    """hpc_rope_norm writing into a block-scaled cache (E4M3 k_cache, v_cache and
    kv_scale [num_pages, Hkv, 2, 4]).  q_scale_out given: E4M3 queries, else BF16."""
    fn, dev = "hpc_rope_norm_block", _current_device()
    Hq, Hkv = int(Hq), int(Hkv)
    (wq_, wk_, pos_, req_, bt_, k_, v_, sc_, q_, qs_, fl_, fr_), shape, count = _arrays(
        fn, dev, "q_norm_w k_norm_w positions token_req block_table k_cache v_cache kv_scale q_out "
        "q_scale_out flags freq", _WRITE_TYPES[q_scale_out is not None], q_norm_w, k_norm_w,
        positions, token_req, block_table, k_cache, v_cache, kv_scale, q_out, q_scale_out, flags,
        freq)
    N, table, pages, rows = count[2], shape[4], shape[5][0] if shape[5] else 0, qkv.shape
    want = (pages, PAGE_SIZE, Hkv, HEAD_DIM)
    _shape(fn, "k_cache", shape[5], want)
    _shape(fn, "v_cache", shape[6], want)
    _shape(fn, "kv_scale", shape[7], (pages, Hkv, 2, PAGE_SIZE // SCALE_BLOCK))
    if qkv.dtype is not _BF16 or len(rows) != 2 or (N and qkv.stride(1) != 1) or rows[0] < N or \
            rows[1] < (Hq + 2 * Hkv) * HEAD_DIM:
        raise ValueError(f"{fn}: qkv is not a BF16 matrix of {N} rows of {Hq} + 2 x {Hkv} heads")
    if qkv.get_device() != dev:
        raise ValueError(f"{fn}: qkv is on {qkv.device}, not on the current device")
    if count[0] != HEAD_DIM or count[1] != HEAD_DIM or \
            (freq is not None and count[11] != HEAD_DIM // 2):
        raise ValueError(f"{fn}: norm weights hold {HEAD_DIM} values, freq {HEAD_DIM // 2}")
    if count[8] < N * Hq * HEAD_DIM or (q_scale_out is not None and count[9] < N * Hq):
        raise ValueError(f"{fn}: q_out or q_scale_out does not hold {N} x {Hq} rows")
    if len(table) != 2 or (token_req is not None and count[3] != N):
        raise ValueError(f"{fn}: block_table is no matrix or token_req has not {N} entries")
    # a stride says nothing where there are not two rows
    stride = qkv.stride(0) if rows[0] > 1 else rows[1]
    params = hpc_rope_norm_params(float(eps), float(rope_base), int(rope_layout),
                                  1 if norm_first else 0, fr_)
    status = lib().hpc_rope_norm_block(
        qkv.data_ptr(), stride, wq_, wk_, pos_, req_, N, Hq, Hkv, HEAD_DIM, bt_,
        table[1], table[0], k_, v_, sc_, pages, q_, qs_, fl_,
        ctypes.byref(params), _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_kv_read_block(k_cache, v_cache, kv_scale, block_table, starts, seqlens, Hkv, k_out, v_out,
                      out_block_table, flags=None, stream=None):
    """Tokens starts[r] .. seqlens[r] - 1 (starts None: from 0) of a block-scaled
    cache as BF16 into the pages out_block_table names."""
    fn, dev, Hkv = "hpc_kv_read_block", _current_device(), int(Hkv)
    (k_, v_, sc_, bt_, st_, sl_, ko_, vo_, ot_, fl_), shape, count = _arrays(
        fn, dev, "k_cache v_cache kv_scale block_table starts seqlens k_out v_out out_block_table "
        "flags", (_E4M3, _E4M3, _F32, _I32, _I32, _I32, _BF16, _BF16, _I32, _I32), k_cache, v_cache,
        kv_scale, block_table, starts, seqlens, k_out, v_out, out_block_table, flags)
    B, pages, out_pages = count[5], *(shape[i][0] if shape[i] else 0 for i in (0, 6))
    want, out_want = (pages, PAGE_SIZE, Hkv, HEAD_DIM), (out_pages, PAGE_SIZE, Hkv, HEAD_DIM)
    _shape(fn, "k_cache", shape[0], want)
    _shape(fn, "v_cache", shape[1], want)
    _shape(fn, "k_out", shape[6], out_want)
    _shape(fn, "v_out", shape[7], out_want)
    _shape(fn, "kv_scale", shape[2], (pages, Hkv, 2, PAGE_SIZE // SCALE_BLOCK))
    _table(fn, "block_table", shape[3], B)
    _table(fn, "out_block_table", shape[8], B)
    if starts is not None and count[4] != B:
        raise ValueError(f"{fn}: starts has not {B} entries")
    status = lib().hpc_kv_read_block(
        k_, v_, sc_, pages, bt_, shape[3][1], st_, sl_, B, Hkv, HEAD_DIM, ko_, vo_, out_pages, ot_,
        shape[8][1], fl_, _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


class SharedWorkspace:
    """The plan and the split buffers of decode steps over shared prefixes, for batches of up
    to num_groups groups of one shape."""

    def __init__(self, B: int, Hq: int, Hkv: int, num_groups: int, *, num_ctas: int = 0,
                 device="cuda", kv_dtype: int = HPC_KV_BF16, q_len: int = 1):
        dev = torch.device(device)
        if num_ctas <= 0:
            num_ctas = hpc_decode_num_ctas(dev.index or 0, kv_dtype)
        sizes = (ctypes.c_int64 * 3)()
        _check("hpc_decode_shared_capacity", lib().hpc_decode_shared_capacity(
            int(B), int(Hq), int(Hkv), int(q_len), int(num_groups), num_ctas, sizes))
        cap, ints, slots = (int(n) for n in sizes)
        self.B, self.Hq, self.Hkv, self.q_len = int(B), int(Hq), int(Hkv), int(q_len)
        self.num_groups, self.num_ctas, self.kv_dtype = int(num_groups), num_ctas, int(kv_dtype)
        self.device = dev
        self.tmap = TaskMap(B, Hkv, cap, num_ctas + 1, dev)
        self.head = torch.zeros(ints, dtype=torch.int32, device=dev)
        rows = q_len * (Hq // Hkv)
        f32 = dict(dtype=torch.float32, device=dev)
        self.part_o = torch.empty((cap, rows, HEAD_DIM), **f32)
        self.part_lse = torch.empty((cap, rows), **f32)
        self.head_o = torch.empty((slots, 128, HEAD_DIM), **f32)
        self.head_lse = torch.empty((slots, 128), **f32)
        self.c = hpc_shared_map(self.tmap.c, _ptr(self.head), _ptr(self.head_o),
                                _ptr(self.head_lse), ints, slots)
        self.tmap.c = self.c.tail  # the planner writes to this one
        _ready(dev)

    @property
    def flags(self) -> int:
        """HPC_FLAG_* bits of the last step (synchronises)."""
        return int(self.tmap.meta[3])

    def head_ctas(self) -> int:
        """CTAs that the last plan gave to the shared pages (synchronises)."""
        return int(self.head[0])


def _groups_arg(fn, starts, groups_shape, ws):
    """The number of groups, checked against the workspace."""
    n = starts[0] - 1 if starts else 0
    if len(starts) != 1 or n < 0 or groups_shape != (n,):
        raise ValueError(f"{fn}: group_starts is no list of one more than prefix_pages")
    if n > ws.num_groups:
        raise ValueError(f"{fn}: {n} groups, but the workspace has room for {ws.num_groups}")
    return n


def hpc_decode_plan_shared(seqlens, group_starts, prefix_pages, Hq, Hkv, q_len, max_pages_per_req,
                           min_tiles_per_cta, ws: SharedWorkspace, stream=None):
    """Plans decode steps of a batch whose groups share their first pages: group g is requests
    group_starts[g] .. group_starts[g + 1] - 1, its pages the first prefix_pages[g]."""
    fn, dev = "hpc_decode_plan_shared", _current_device()
    (sl_, gs_, pp_), shape, count = _arrays(fn, dev, "seqlens group_starts prefix_pages",
                                            (_I32, _I32, _I32), seqlens, group_starts,
                                            prefix_pages)
    _on(fn, ws, dev)
    n = _groups_arg(fn, shape[1], shape[2], ws)
    _check(fn, lib().hpc_decode_plan_shared(
        sl_, count[0], int(Hq), int(Hkv), int(max_pages_per_req), gs_, pp_, n, ws.num_ctas,
        int(min_tiles_per_cta), ws.kv_dtype, int(q_len), ctypes.byref(ws.c),
        _raw_stream(dev, stream)))


def _on(fn, ws, dev):
    if not isinstance(ws, SharedWorkspace) or ws.head.get_device() != dev:
        raise ValueError(f"{fn}: no SharedWorkspace on the current device")


def hpc_decode_attn_shared(q, q_scale, k_cache, v_cache, k_scale, v_scale, kv_scale, block_table,
                           seqlens, Hq, Hkv, q_len, sm_scale, ws: SharedWorkspace, out,
                           stream=None):
    """Attention of a batch that hpc_decode_plan_shared planned, as hpc_decode_step_mq
    computes it.  kv_scale: the block scales of a block-scaled cache, else None."""
    fn = "hpc_decode_attn_shared"
    _on(fn, ws, _current_device())
    Hq, Hkv, q_len = int(Hq), int(Hkv), int(q_len)
    kv, dev, B, pages, cols, (q_, k_, v_, qs_, sc_, bt_, sl_, po_, pl_, _, out_) = _win_args(
        fn, q, q_scale, k_cache, v_cache, kv_scale, block_table, seqlens, Hq, Hkv, q_len,
        ws.part_o, ws.part_lse, out, None, ws.tmap.cap_desc)
    status = lib().hpc_decode_attn_shared(
        q_, qs_, k_, v_, pages, float(k_scale), float(v_scale), sc_, kv, bt_, cols, sl_, B, Hq,
        Hkv, HEAD_DIM, q_len, float(sm_scale), ctypes.byref(ws.c), po_, pl_, out_,
        _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_decode_step_shared(q, q_scale, k_cache, v_cache, k_scale, v_scale, kv_scale, block_table,
                           seqlens, group_starts, prefix_pages, Hq, Hkv, q_len, sm_scale,
                           min_tiles_per_cta, ws: SharedWorkspace, out, stream=None):
    """hpc_decode_plan_shared and hpc_decode_attn_shared in one call."""
    fn = "hpc_decode_step_shared"
    _on(fn, ws, _current_device())
    Hq, Hkv, q_len = int(Hq), int(Hkv), int(q_len)
    kv, dev, B, pages, cols, (q_, k_, v_, qs_, sc_, bt_, sl_, po_, pl_, _, out_) = _win_args(
        fn, q, q_scale, k_cache, v_cache, kv_scale, block_table, seqlens, Hq, Hkv, q_len,
        ws.part_o, ws.part_lse, out, None, ws.tmap.cap_desc)
    (gs_, pp_), shape, _ = _arrays(fn, dev, "group_starts prefix_pages", (_I32, _I32),
                                   group_starts, prefix_pages)
    n = _groups_arg(fn, shape[0], shape[1], ws)
    status = lib().hpc_decode_step_shared(
        q_, qs_, k_, v_, pages, float(k_scale), float(v_scale), sc_, kv, bt_, cols, sl_, gs_, pp_,
        n, B, Hq, Hkv, HEAD_DIM, q_len, float(sm_scale), ws.num_ctas, int(min_tiles_per_cta),
        ctypes.byref(ws.c), po_, pl_, out_, _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


class PagePool:
    """The pages of a cache: how many table entries name each (refs), a stack of those that
    none names (free_list) and the state {pages on the stack, flags, 0, 0}."""

    def __init__(self, num_pages: int, device="cuda"):
        dev = torch.device(device)
        self._of(torch.zeros(num_pages, dtype=torch.int32, device=dev),
                 torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=dev),
                 torch.tensor([num_pages, 0, 0, 0], dtype=torch.int32, device=dev))

    @classmethod
    def of(cls, refs, free_list, state):
        """A pool on arrays that say which pages are held already."""
        self = cls.__new__(cls)
        self._of(refs, free_list, state)
        return self

    def _of(self, refs, free_list, state):
        self.num_pages = int(refs.numel())
        if any(t.dtype is not _I32 or not t.is_contiguous() or t.device != refs.device
               for t in (refs, free_list, state)) or free_list.numel() != self.num_pages or \
                state.numel() != 4:
            raise ValueError("PagePool: refs, free_list [num_pages] and state [4] are int32 "
                             "arrays of one device")
        self.refs, self.free_list, self.state = refs, free_list, state
        self.marks = torch.full_like(refs, 2 ** 31 - 1)
        self.c = hpc_page_pool(_ptr(refs), _ptr(free_list), _ptr(state), _ptr(self.marks),
                               self.num_pages)
        self.ref, self.dev = ctypes.byref(self.c), refs.get_device()
        _ready(refs.device)

    @property
    def free_pages(self) -> int:
        """Pages on the stack (synchronises)."""
        return int(self.state[0])

    @property
    def flags(self) -> int:
        """HPC_FLAG_* bits raised so far (synchronises)."""
        return int(self.state[1])


_I32S = [(_I32,) * n for n in range(6)]


def _pool_table(fn, dev, pool, shape):
    """The table's rows and columns; raises for a pool of another device or no pool."""
    if type(pool) is not PagePool or pool.dev != dev:
        raise ValueError(f"{fn}: no PagePool on the current device")
    if len(shape) != 2:
        raise ValueError(f"{fn}: block_table is no matrix")
    return shape


def _listed(fn, name, n):
    raise ValueError(f"{fn}: {name} has not {n} entries")


def _cap(fn, shape):
    if len(shape) != 2 or shape[0] < 1 or shape[1] != 2:
        raise ValueError(f"{fn}: copies is {shape}, not [1 + capacity, 2]")
    return shape[0] - 1


def hpc_kv_free(pool: PagePool, block_table, rows=None, keep=None, stream=None):
    """The rows (None: all) give back the pages behind their first keep[i] tokens (None: all).
    A shared page that keep ends inside stays shared: to write there, fork and free the row."""
    fn, dev = "hpc_kv_free", _current_device()
    adr, shape, count = _arrays(fn, dev, "block_table rows keep", _I32S[3], block_table, rows, keep)
    B, cols = _pool_table(fn, dev, pool, shape[0])
    n = B if rows is None else count[1]
    if keep is not None and count[2] != n:
        _listed(fn, "keep", n)
    status = lib().hpc_kv_free(pool.ref, adr[0], B, cols, adr[1], adr[2], n,
                               _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_kv_extend(pool: PagePool, block_table, rows, lens, stream=None):
    """The rows (None: all) get the pages that lens[i] tokens need and they have not."""
    fn, dev = "hpc_kv_extend", _current_device()
    adr, shape, count = _arrays(fn, dev, "block_table rows lens", _I32S[3], block_table, rows, lens)
    B, cols = _pool_table(fn, dev, pool, shape[0])
    n = B if rows is None else count[1]
    if count[2] != n:
        _listed(fn, "lens", n)
    status = lib().hpc_kv_extend(pool.ref, adr[0], B, cols, adr[1], adr[2], n,
                                 _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_kv_fork(pool: PagePool, block_table, src, dst, lens, copies, stream=None):
    """Row dst[i] becomes a fork of the first lens[i] tokens of row src[i]; copies [1 + cap, 2]
    gets the pages to copy ({count, 0}, then {from, to})."""
    fn, dev = "hpc_kv_fork", _current_device()
    adr, shape, count = _arrays(fn, dev, "block_table src dst lens copies", _I32S[5], block_table,
                                src, dst, lens, copies)
    B, cols = _pool_table(fn, dev, pool, shape[0])
    if None in count:
        raise ValueError(f"{fn}: src, dst, lens and copies are needed")
    n = count[1]
    if count[2] != n or count[3] != n:
        _listed(fn, "dst" if count[2] != n else "lens", n)
    status = lib().hpc_kv_fork(pool.ref, adr[0], B, cols, adr[1], adr[2], adr[3], n, adr[4],
                               _cap(fn, shape[4]), _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


def hpc_kv_compact(pool: PagePool, block_table, copies, out_table=None, out_pool=None,
                   stream=None):
    """The pages that are held move into the first places; copies [1 + cap, 2] gets the moves.
    out_table, out_pool: where the table and the pool are written (None: in place)."""
    fn, dev = "hpc_kv_compact", _current_device()
    if out_table is None:
        out_table = block_table
    if out_pool is None:
        out_pool = pool
    adr, shape, count = _arrays(fn, dev, "block_table copies out_table", _I32S[3], block_table,
                                copies, out_table)
    B, cols = _pool_table(fn, dev, pool, shape[0])
    _pool_table(fn, dev, out_pool, shape[0])
    if copies is None:
        raise ValueError(f"{fn}: copies is needed")
    if shape[2] != shape[0]:
        _shape(fn, "out_table", shape[2], shape[0])
    status = lib().hpc_kv_compact(pool.ref, adr[0], B, cols, adr[1], _cap(fn, shape[1]), adr[2],
                                  out_pool.ref, _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


_PAGE_TYPES = [(_I32, t, t, _F32, _I32) for t in (_BF16, _E4M3)]


def hpc_kv_copy_pages(copies, k_cache, v_cache, kv_scale=None, flags=None, stream=None):
    """The copies that hpc_kv_fork or hpc_kv_compact listed, in one layer's caches (and the
    block scales [num_pages, Hkv, 2, 4] of a block-scaled one)."""
    fn, dev = "hpc_kv_copy_pages", _current_device()
    e4m3 = k_cache is not None and k_cache.dtype is _E4M3
    adr, shape, _ = _arrays(fn, dev, "copies k_cache v_cache kv_scale flags", _PAGE_TYPES[e4m3],
                            copies, k_cache, v_cache, kv_scale, flags)
    cache = shape[1]
    if copies is None or cache is None or len(cache) != 4:
        raise ValueError(f"{fn}: copies, or a cache [num_pages, 64, Hkv, 128]")
    pages, Hkv = cache[0], cache[2]
    if cache[1] != PAGE_SIZE or cache[3] != HEAD_DIM:
        _shape(fn, "k_cache", cache, (pages, PAGE_SIZE, Hkv, HEAD_DIM))
    if shape[2] != cache:
        _shape(fn, "v_cache", shape[2], cache)
    kv = HPC_KV_FP8_E4M3 if e4m3 else HPC_KV_BF16
    if kv_scale is not None:
        if not e4m3:
            raise ValueError(f"{fn}: kv_scale belongs to E4M3 pages")
        _shape(fn, "kv_scale", shape[3], (pages, Hkv, 2, PAGE_SIZE // SCALE_BLOCK))
        kv = HPC_KV_E4M3_BLOCK
    status = lib().hpc_kv_copy_pages(adr[0], _cap(fn, shape[0]), adr[1], adr[2], adr[3], kv, pages,
                                     Hkv, HEAD_DIM, adr[4], _raw_stream(dev, stream))
    if status != HPC_OK:
        _check(fn, status)


class Workspace:
    """Split buffer, output and task map sized for one batch shape, for the plain and the
    windowed calls over kv_dtype caches."""

    def __init__(self, B: int, Hq: int, Hkv: int, *, num_ctas: int = 0, num_splits: int = 0,
                 device="cuda", kv_dtype: int = HPC_KV_BF16, q_len: int = 1):
        dev = torch.device(device)
        if num_splits:
            self.tmap = TaskMap.static(B, Hkv, num_splits, dev)
        else:
            if num_ctas <= 0:
                num_ctas = hpc_decode_num_ctas(dev.index or 0, kv_dtype)
            # descriptors of head pairs (the _win calls, over 8-bit caches of an even
            # number of heads) need more room
            pairs = 2 if kv_dtype != HPC_KV_BF16 and Hkv % 2 == 0 else 1
            cap = hpc_decode_desc_capacity(B, Hkv, pairs * num_ctas)
            self.tmap = TaskMap(B, Hkv, cap, num_ctas + 1, dev)
        self.num_ctas, self.num_splits = num_ctas, num_splits
        rows = q_len * (Hq // Hkv)  # query rows of one KV head in a descriptor
        cap = max(self.tmap.cap_desc, 1)
        self.q_len = q_len
        self.part_o = torch.empty((cap, rows, HEAD_DIM), dtype=torch.float32, device=dev)
        self.part_lse = torch.empty((cap, rows), dtype=torch.float32, device=dev)
        out_shape = (max(B, 1), Hq, HEAD_DIM) if q_len == 1 else (max(B, 1), q_len, Hq, HEAD_DIM)
        self.out = torch.empty(out_shape, dtype=torch.bfloat16, device=dev)
        # chunk counters of the fused combine: zero once, left zero by every launch
        self.unit_done = torch.zeros(max(B * Hkv, 1), dtype=torch.int32, device=dev)
        _ready(dev)
