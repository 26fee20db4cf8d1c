"""Planners called by several host threads at once, for batches of different sizes whose
lengths do not fit the 48 KB of shared memory that a launch gets unasked."""

import ctypes
import threading

import pytest
import torch

import load_balanced_paged_assign_gb300 as hd

pytestmark = pytest.mark.gpu

CALLS = 10000


def together(calls):
    """Each call (of the library, so that the threads run at once) CALLS times in a thread of
    its own, on a stream of its own; the statuses that were not HPC_OK."""
    failed, start = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        handle = ctypes.c_void_p(stream.cuda_stream)
        start.wait()
        failed.extend(s for s in (call(handle) for _ in range(CALLS)) if s != 0)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


def lengths(B):
    return (torch.arange(B, device="cuda", dtype=torch.int32) * 37) % 128 + 1


def test_plans_of_shared_prefixes():
    plans = [(hd.SharedWorkspace(B, 1, 1, 0), lengths(B)) for B in (8192, 6000, 4200)]
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    fn = hd.lib().hpc_decode_plan_shared

    def call_of(ws, lens):
        args = (lens.data_ptr(), lens.numel(), 1, 1, 2, starts.data_ptr(), None, 0, ws.num_ctas, 2,
                0, 1, ctypes.byref(ws.c))
        return lambda handle: fn(*args, handle)

    assert together([call_of(*p) for p in plans]) == []
    for ws, lens in plans:
        assert ws.flags == 0 and int(ws.tmap.meta[0]) == int(((lens + 63) // 64).sum())


@pytest.mark.parametrize("window", [0, 64])
def test_plans(window):
    plans = [(hd.TaskMap.dynamic(B, 1, 152), lengths(B)) for B in (16384, 14500, 12800)]
    fn = hd.lib().hpc_decode_plan_win

    def call_of(tmap, lens):
        args = (lens.data_ptr(), lens.numel(), 1, 2, 152, 2, 0, 1, window, 0, ctypes.byref(tmap.c))
        return lambda handle: fn(*args, handle)

    assert together([call_of(*p) for p in plans]) == []
    for tmap, lens in plans:
        got = tmap.to_host()
        assert got["flags"] == 0
        if not window:
            assert got["total_tiles"] == int(((lens + 63) // 64).sum())
