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


# addresses far apart, and sizes of a layer of 4 tokens, 8 experts of 128 x 256 and a shared one
AT = [n << 32 for n in range(1, 20)]
HUGE = 1 << 30


def _few(moe, fmt, y, ws):
    """A call of one of the three forms; y and the workspace lie where the caller says."""
    s = moe.make_shape(4, 128, 8, 2, 256, 128, "bf16")
    names = ["moe_forward_few", "moe_forward_few_fp8", "moe_forward_few_fp8_blocks"]
    call = getattr(moe.library(), names[fmt])
    if fmt == 0:
        return call(ctypes.byref(s), AT[0], AT[1], ctypes.c_void_p(AT[2]), *AT[3:9], AT[9], y, ws, HUGE, None)
    w = moe.moe_fp8_experts(*AT[3:6], *AT[10:13], *AT[6:9], *AT[13:16])
    return call(ctypes.byref(s), AT[0], AT[1], ctypes.c_void_p(AT[2]), ctypes.byref(w), AT[9], y, ws, HUGE,
                None)


def _few_reads(fmt):
    """(address, bytes) of what the call reads, the residual (AT[9]) apart"""
    E, d, I, Is, size = 8, 128, 256, 128, 2 if fmt == 0 else 1  # noqa: E741
    out = [(AT[0], 4 * d * 2), (AT[1], E * d * 2), (AT[2], 4 * E)]
    out += [(AT[i], E * I * d * size) for i in (3, 4, 5)] + [(AT[i], Is * d * size) for i in (6, 7, 8)]
    if fmt == 1:
        out += [(AT[10], 4 * E * I), (AT[11], 4 * E * I), (AT[12], 4 * E * d)]
        out += [(AT[13], 4 * Is), (AT[14], 4 * Is), (AT[15], 4 * d)]
    if fmt == 2:
        out += [(AT[i], 4 * E * 2) for i in (10, 11, 12)] + [(AT[i], 4) for i in (13, 14, 15)]
    return out


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_few_tokens_write_nothing_that_they_read(moe, fmt):
    """y and the workspace apart from every input, and from one another."""
    rows, ws = 4 * 128 * 2, moe.moe_few_workspace_bytes(moe.make_shape(4, 128, 8, 2, 256, 128, "bf16"))
    for at, n in _few_reads(fmt):
        last = at + (n - 1) // 16 * 16  # the last 16-byte boundary inside
        for y in (at, last, at - rows + 16):
            assert _few(moe, fmt, y, AT[17]) == 1, (at, y)
        for w in (at, last):
            assert _few(moe, fmt, AT[16], w) == 1, (at, w)
    assert _few(moe, fmt, AT[9] + 16, AT[17]) == 1
    assert _few(moe, fmt, AT[16], AT[9]) == 1
    assert _few(moe, fmt, AT[17] + ws // 2 // 16 * 16, AT[17]) == 1


def test_backward_workspace_apart_from_the_arrays(moe):
    back = moe.library().moe_rmsnorm_backward
    need = moe.moe_rmsnorm_workspace_bytes(40, 64)
    args = dict(dy=AT[0], s=AT[1], w=AT[2], ds=AT[3], dx=AT[4], dw=AT[5])
    for name, at in args.items():
        for ws in (at, at - need + 256, at + 16):
            assert back(40, 64, 1, args["dy"], args["s"], args["w"], 1e-6, args["ds"], args["dx"], args["dw"],
                        ws, HUGE, None) == 1, name
