"""Calls of the norm and of the layer for a few tokens at the edge of what they take."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_an_empty_batch(moe, dtype):
    """The norm and its gradients of no rows: nothing is written but a weight's gradient of zeros."""
    x, w = torch.empty(0, 64, dtype=dtype, device="cuda"), torch.ones(64, dtype=dtype, device="cuda")
    codes = torch.empty(0, 64, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm(x, None, w, 1e-6, None, torch.empty_like(x), codes, torch.empty(0, device="cuda"))
    ws = moe.alloc_rmsnorm_workspace(0, 64)
    for d_weight in (None, torch.ones(64, device="cuda")):
        for d_x in (None, torch.empty_like(x)):
            moe.moe_rmsnorm_backward(x, x, w, 1e-6, x, d_x, d_weight, ws)
            if d_weight is not None:
                assert (d_weight == 0).all()
                d_weight.fill_(1)
