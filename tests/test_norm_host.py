"""The norm's calls refuse bad arguments on the host, and its plain statement is that of
torch's autograd (no GPU needed)."""
import ctypes

import pytest
import torch

from tests import norm_ref as ref


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import sparse_expert_ffn_moe_gb300 as m
    return m


A, B, C, D, E = (ctypes.c_void_p(1 << n) for n in (32, 33, 34, 35, 36))
ODD = ctypes.c_void_p((1 << 32) + 8)
NAN, INF = float("nan"), float("inf")


def _norm(moe, rows=4, cols=64, dtype=1, x=A, r=None, w=B, eps=1e-6, s=None, y=C, codes=None,
          scales=None):
    return moe.library().moe_rmsnorm(rows, cols, dtype, x, r, w, eps, s, y, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=2), 1), (dict(cols=16385), 2),
    (dict(rows=1 << 31), 2), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(eps=-1e-6), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(x=ODD), 1), (dict(y=ODD), 1),
    (dict(codes=D), 1), (dict(scales=D), 1), (dict(s=A, y=A), 1), (dict(s=B), 1), (dict(y=B), 1),
    (dict(r=D, y=D), 1), (dict(y=ctypes.c_void_p((1 << 32) + 16)), 1),
    (dict(codes=A, scales=D), 1), (dict(codes=D, scales=D), 1)])
def test_norm_refusals(moe, kw, status):
    assert _norm(moe, **kw) == status


def test_no_rows_is_a_no_op(moe):
    assert _norm(moe, rows=0, x=None, w=None, y=None) == 0


def _back(moe, rows=4, cols=64, dtype=1, dy=A, s=B, w=C, eps=1e-6, ds=None, dx=D, dw=None, ws=None,
          n=0):
    return moe.library().moe_rmsnorm_backward(rows, cols, dtype, dy, s, w, eps, ds, dx, dw, ws, n,
                                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=-1), 1), (dict(cols=16385), 2),
    (dict(eps=NAN), 1), (dict(dy=None), 1), (dict(s=None), 1), (dict(w=None), 1),
    (dict(dx=None), 1), (dict(dx=ODD), 1), (dict(ds=ODD), 1), (dict(dx=C), 1),
    (dict(dx=ctypes.c_void_p((1 << 32) + 32)), 1), (dict(dw=E), 3), (dict(dw=E, ws=A, n=16), 3),
    (dict(dw=A, ws=E, n=1 << 30), 1), (dict(dw=D, ws=E, n=1 << 30), 1)])
def test_backward_refusals(moe, kw, status):
    assert _back(moe, **kw) == status


def test_workspace_sizes(moe):
    assert moe.moe_rmsnorm_workspace_bytes(-1, 8) == 0
    assert moe.moe_rmsnorm_workspace_bytes(8, 16385) == 0
    assert moe.moe_rmsnorm_workspace_bytes(16384, 7168) >= 4 * 7168
    with pytest.raises(moe.MoeError):
        moe.alloc_rmsnorm_workspace(4, 0)


def test_binding_refuses_host_tensors_and_other_types(moe):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm(x, None, torch.zeros(8), 1e-6, None, x, None, None)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm(x.half(), None, torch.zeros(8), 1e-6, None, x, None, None)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm_backward(x, x.half(), torch.zeros(8), 1e-6, None, x, None, None)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_statement_is_autograd(eps):
    g = torch.Generator().manual_seed(1)
    s = torch.randn(9, 33, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    dy, ds = (torch.randn(9, 33, generator=g, dtype=torch.float64) for _ in range(2))
    y = torch.nn.functional.rms_norm(s, (33,), w, eps)
    assert torch.allclose(ref.norm(s, w, eps), y, rtol=1e-13)
    dx, dw = torch.autograd.grad(y, (s, w), dy)
    a, _, b, _ = ref.grads(dy, s, w, eps, ds)
    assert torch.allclose(a, dx + ds, rtol=1e-12) and torch.allclose(b, dw, rtol=1e-12)
