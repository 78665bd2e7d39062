"""Launches whose shared memory passes the 48 KB that a launch has without asking for more."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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
