"""The calls for a few tokens refuse bad arguments on the host (no GPU needed), and their
plain 64-bit statement is the oracle's layer."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from tests import few_ref as ref


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import sparse_expert_ffn_moe_gb300 as m
    return m


P = [ctypes.c_void_p(1 << n) for n in range(32, 46)]
ODD = ctypes.c_void_p((1 << 32) + 8)
HUGE = 1 << 40


def _call(moe, shape=(4, 128, 8, 2, 128, 128, "bf16"), x=P[0], w_g=P[1], bias=None, gate=P[2],
          up=P[3], down=P[4], sg=P[5], su=P[6], sd=P[7], residual=None, y=P[8], ws=P[9], n=HUGE):
    s = moe.make_shape(*shape)
    return moe.library().moe_forward_few(ctypes.byref(s), x, w_g, bias, gate, up, down, sg, su, sd,
                                         residual, y, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(shape=(17, 128, 8, 2, 128, 128, "bf16")), 2), (dict(shape=(4, 128, 8, 2, 128, 128, "f32")), 2),
    (dict(shape=(4, 100, 8, 2, 128, 128, "bf16")), 2), (dict(shape=(4, 128, 2, 8, 128, 128, "bf16")), 1),
    (dict(shape=(-1, 128, 8, 2, 128, 128, "bf16")), 1), (dict(x=None), 1), (dict(w_g=None), 1),
    (dict(gate=None), 1), (dict(down=ODD), 1), (dict(sg=None), 1), (dict(y=None), 1), (dict(y=ODD), 1),
    (dict(bias=ctypes.c_void_p((1 << 32) + 2)), 1), (dict(residual=ODD), 1), (dict(y=P[0]), 1),
    (dict(y=ctypes.c_void_p((1 << 32) + 64)), 1),
    (dict(residual=ctypes.c_void_p(P[8].value + 16)), 1),
    (dict(shape=(4, 128, 8, 2, 128, 0, "bf16")), 1),  # shared weights without a shared expert
    (dict(ws=None), 3), (dict(n=1024), 3), (dict(ws=ODD), 3)])
def test_refusals(moe, kw, status):
    assert _call(moe, **kw) == status


def test_no_tokens_is_a_no_op(moe):
    assert _call(moe, shape=(0, 128, 8, 2, 128, 128, "bf16"), x=None, y=None, ws=None) == 0


def _call8(moe, shape=(4, 128, 8, 2, 128, 0, "bf16"), drop=(), n=HUGE, shared=False, name="moe_forward_few_fp8"):
    s = moe.make_shape(*shape)
    fields = [f for f, _ in moe.moe_fp8_experts._fields_]
    w = moe.moe_fp8_experts(*[None if f in drop or (not shared and f[1] == "s") else 1 << 33
                              for f in fields])
    return getattr(moe.library(), name)(ctypes.byref(s), P[0], P[2], None, ctypes.byref(w), None, P[8],
                                        P[9], n, None)


@pytest.mark.parametrize("name", ["moe_forward_few_fp8", "moe_forward_few_fp8_blocks"])
def test_refusals_8_bit(moe, name):
    assert _call8(moe, shape=(4, 192, 8, 2, 128, 0, "bf16"), name=name) == 2
    assert _call8(moe, shape=(4, 128, 8, 2, 64, 0, "bf16"), name=name) == 2
    assert _call8(moe, shape=(17, 128, 8, 2, 128, 0, "bf16"), name=name) == 2
    for f in ("w_gate", "s_up", "s_down"):
        assert _call8(moe, drop=(f,), name=name) == 1
    assert _call8(moe, shared=True, name=name) == 1  # shared codes without a shared expert
    assert _call8(moe, shape=(4, 128, 8, 2, 128, 128, "bf16"), shared=True, drop=("ss_down",),
                  name=name) == 1
    assert _call8(moe, n=256, name=name) == 3
    null = ctypes.POINTER(moe.moe_fp8_experts)()
    s = moe.make_shape(4, 128, 8, 2, 128, 0, "bf16")
    assert getattr(moe.library(), name)(ctypes.byref(s), P[0], P[2], None, null, None, P[8], P[9],
                                        HUGE, None) == 1


def test_workspace_sizes(moe):
    assert moe.moe_few_workspace_bytes(moe.make_shape(17, 128, 8, 2, 128, 0)) == 0
    assert moe.moe_few_workspace_bytes(moe.make_shape(4, 128, 2, 8, 128, 0)) == 0
    small = moe.moe_few_workspace_bytes(moe.make_shape(1, 256, 8, 2, 512, 0))
    assert 0 < small < moe.moe_few_workspace_bytes(moe.make_shape(16, 7168, 256, 8, 2048, 2048))
    with pytest.raises(moe.MoeError):
        moe.alloc_few_workspace(moe.make_shape(17, 128, 8, 2, 128, 0))


def test_binding_refuses_wrong_tensors(moe):
    s = moe.make_shape(1, 128, 2, 1, 128, 0)
    x = torch.zeros(1, 128)
    with pytest.raises(ValueError):
        moe.moe_forward_few(s, x, x, None, x, x, x, None, None, None, None, x, None)


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_statement_is_the_oracles_layer(router):
    c = ref.inputs(5, 128, 12, 3, 64, 128, router, "bf16", 1)
    want, tol = ref.layer(c)
    f = {k: v.float().numpy() for k, v in c.items() if torch.is_tensor(v)}
    out = oracle.forward_tokens(np.arange(5), f["x"], f, 3, bias=f["bias"], router=router)
    y = out["y"] + f["residual"].astype(np.float64)
    assert np.abs(y - want.numpy()).max() < 1e-6 * np.abs(want.numpy()).max()
    assert (tol > 0).all()
