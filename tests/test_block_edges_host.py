"""Calls of the norm and of the layer for a few tokens at the edge of what they take, on the host
(no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import sparse_expert_ffn_moe_gb300 as m
    return m


def test_no_rows_have_a_workspace(moe):
    """An empty batch is a valid call, so its workspace can be asked for."""
    for cols in (1, 64, 16384):
        assert moe.moe_rmsnorm_workspace_bytes(0, cols) > 0
    assert moe.alloc_rmsnorm_workspace(0, 64, device="cpu").numel() > 0
    assert moe.moe_rmsnorm_workspace_bytes(0, 0) == 0


def test_no_rows_and_no_arrays(moe):
    """What has no elements has no address: d_x of an empty batch is NULL."""
    back = moe.library().moe_rmsnorm_backward
    assert back(0, 64, 1, None, None, None, 1e-6, None, None, None, None, 0, None) == 0
    assert back(1, 64, 1, None, None, None, 1e-6, None, None, None, None, 0, None) == 1
    assert back(0, 64, 1, None, None, None, 1e-6, None, ctypes.c_void_p(8), None, None, 0, None) == 1
