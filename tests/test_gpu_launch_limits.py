"""Launches whose shared memory passes the 48 KB that a launch has without asking for more."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


# The norm's backward pass with rings of 48 KB, just below and above: the limit counts the
# kernel's static arrays too.  A process of their own: a wider call before them would have asked.
FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
import sparse_expert_ffn_moe_gb300 as moe
for d, t in {sizes!r}:
    t = getattr(torch, t)
    x, w = torch.ones(5, d, dtype=t, device="cuda"), torch.ones(d, dtype=t, device="cuda")
    dx, dw = torch.full_like(x, 9), torch.full((d,), 9.0, device="cuda")
    moe.moe_rmsnorm_backward(x, x, w, 0.0, None, dx, dw, moe.alloc_rmsnorm_workspace(5, d))
    torch.cuda.synchronize()
    # rows of ones: y = x, d_x = 0 but for r's rounding, d_weight = 5
    assert dx.float().abs().max().item() < 1e-5 and (dw - 5).abs().max().item() < 1e-5, d
print("fine")
"""


@pytest.mark.parametrize("sizes", [
    [(4096, "bfloat16"), (4085, "bfloat16"), (2048, "float32"), (2043, "float32")],
    [(4056, "bfloat16"), (4041, "bfloat16"), (2028, "float32"), (2021, "float32")],
    [(4048, "bfloat16"), (4104, "bfloat16"), (2024, "float32"), (2052, "float32")]])
def test_first_call_at_48_kb_of_ring(sizes):
    done = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, sizes=sizes)],
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout == "fine\n", done.stderr[-2000:]


def _side_by_side(calls, n):
    """Every call n times in a host thread of its own, all at once; what they return but 0."""
    wrong = []

    def go(call):
        for _ in range(n):
            rc = call()
            if rc:
                wrong.append(rc)

    threads = [threading.Thread(target=go, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return wrong


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def test_threads_whose_rings_differ_in_size(moe):
    """Calls of several host threads, each on its own stream, of one kernel with rings of
    different sizes: none may lower the limit that another's launch needs."""
    keep, calls = [], []
    for d in (4104, 4608, 5000, 5120):
        x, w = torch.ones(2, d, device="cuda").bfloat16(), torch.ones(d, device="cuda").bfloat16()
        dx, dw, ws = torch.empty_like(x), torch.empty(d, device="cuda"), moe.alloc_rmsnorm_workspace(2, d)
        st = torch.cuda.Stream()
        args = (2, d, moe.MOE_BF16, _ptr(x), _ptr(x), _ptr(w), 0.0, None, _ptr(dx), _ptr(dw), _ptr(ws),
                ws.numel(), ctypes.c_void_p(st.cuda_stream))
        keep.append((x, w, dx, dw, ws, st))
        calls.append(lambda args=args: moe.library().moe_rmsnorm_backward(*args))
    torch.cuda.synchronize()
    assert not _side_by_side(calls, 20000)


# d, E of fp32 layers (rows of x in shared memory), of 8-bit ones (the same as halves), and of
# layers whose dispatch holds a table of experts
LAYERS = {"f32": [(7168, 4), (8192, 4), (16384, 4)], "fp8": [(2048, 4), (4096, 4), (8192, 4)],
          "experts": [(64, 16), (64, 500), (64, 1024)]}


@pytest.mark.parametrize("kind", LAYERS)
def test_threads_whose_layers_differ_in_size(moe, kind):
    keep, calls = [], []
    for d, E in LAYERS[kind]:
        I = 64 if kind == "experts" else 128  # noqa: E741
        s = moe.make_shape(1, d, E, 1, I, 0, "f32" if kind == "f32" else "bf16")
        t = torch.float32 if kind == "f32" else torch.bfloat16
        x, w_g, gate, up = (torch.randn(n, device="cuda").to(t) for n in
                            ((1, d), (E, d), (E, I, d), (E, I, d)))
        down, y, ws = torch.randn(E, d, I, device="cuda").to(t), torch.empty_like(x), moe.alloc_workspace(s)
        st = torch.cuda.Stream()
        tail = (_ptr(y), _ptr(ws), ws.numel(), ctypes.c_void_p(st.cuda_stream))
        if kind == "fp8":
            q = {}
            for n, w in (("gate", gate), ("up", up), ("down", down)):
                q["w_" + n] = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
                q["s_" + n] = torch.empty(w.shape[:-1], device="cuda")
                moe.moe_quantize_fp8_rows(w, q["w_" + n], q["s_" + n])
            w8 = moe.make_fp8_experts(q)
            args = (ctypes.byref(s), _ptr(x), _ptr(w_g), None, ctypes.byref(w8), *tail)
            call = moe.library().moe_forward_fp8
            keep.append((q, w8))
        else:
            args = (ctypes.byref(s), _ptr(x), _ptr(w_g), None, _ptr(gate), _ptr(up), _ptr(down), None, None,
                    None, *tail)
            call = moe.library().moe_forward
        keep.append((s, x, w_g, gate, up, down, y, ws, st))
        calls.append(lambda args=args, call=call: call(*args))
    torch.cuda.synchronize()
    assert not _side_by_side(calls, 3000)
