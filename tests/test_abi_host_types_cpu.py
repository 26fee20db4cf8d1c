"""The host-buffer step and cache types it does not take (no GPU)."""

import ctypes

import pytest

import load_balanced_paged_assign_gb300 as hd
from load_balanced_paged_assign_gb300 import binding as E
from test_abi_window_cpu import FAKE, fake_map


@pytest.mark.parametrize("kv", [E.HPC_KV_E4M3_BLOCK, 3, -1])
def test_the_host_step_refuses_before_it_copies(kv):
    """The block-scaled type has one-byte queries: taken for BF16's, twice the caller's
    buffer would be read.  (Host buffers of one byte: nothing may be read from them.)"""
    from load_balanced_paged_assign_gb300 import _build
    _build.build()
    h = ctypes.cast(ctypes.create_string_buffer(1), ctypes.c_void_p)
    m = fake_map()
    assert hd.lib().hpc_decode_step_host(
        h, h, h, h, h, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 10, 1.0, 1.0, kv, 4, 4, 8, 1, 128,
        0.088, 132, 2, 0, ctypes.byref(m), FAKE, FAKE, FAKE, None) == E.HPC_ERR_ARG
