"""What a constructor makes is ready for calls on any stream when it returns."""

import pytest
import torch

import load_balanced_paged_assign_gb300 as hd

pytestmark = pytest.mark.gpu

MAKE = {
    "TaskMap": lambda: hd.TaskMap.dynamic(40, 8, 152),
    "Workspace": lambda: hd.Workspace(40, 64, 8),
    "SharedWorkspace": lambda: hd.SharedWorkspace(40, 64, 8, 5),
    "PagePool": lambda: hd.PagePool(5000),
    "PagePool.of": lambda: hd.PagePool.of(torch.zeros(5000, dtype=torch.int32, device="cuda"),
                                          torch.arange(5000, dtype=torch.int32, device="cuda"),
                                          torch.zeros(4, dtype=torch.int32, device="cuda")),
}


def keep_busy():
    """Tens of milliseconds of work on the current stream."""
    torch.cuda._sleep(10 ** 8)


@pytest.mark.parametrize("name", MAKE)
@pytest.mark.parametrize("side", [False, True])
def test_nothing_is_pending_when_a_constructor_returns(name, side):
    """Neither its own fills nor, on the stream that the allocator orders them by, what used
    the memory before."""
    with torch.cuda.stream(torch.cuda.Stream() if side else torch.cuda.current_stream()):
        MAKE[name]()  # (its memory is then the allocator's to give again)
        torch.cuda.synchronize()
        keep_busy()
        assert not torch.cuda.current_stream().query()
        made = MAKE[name]()
        assert torch.cuda.current_stream().query()
        del made


def test_constructors_while_a_graph_is_captured():
    """They are part of the graph then, and wait for nothing."""
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        ws = hd.SharedWorkspace(4, 8, 1, 1, num_ctas=152)
        lens = torch.full((4,), 100, dtype=torch.int32, device="cuda")
        starts = torch.zeros(1, dtype=torch.int32, device="cuda")
        hd.hpc_decode_plan_shared(lens, starts, starts[:0], 8, 1, 1, 2, 2, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert ws.flags == 0 and int(ws.tmap.meta[0]) == 8
