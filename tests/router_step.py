"""The joined training step of a router in 64 bits, from what the step's kernels read
(the expert rows and the output's gradient as stored, in bf16), so that fp32 errors
alone are left; and how far the library's gradients may be off.  Tests on the CPU show
that the bounds tell a missing part from rounding; tests on the GPU hold the step to
them."""
from __future__ import annotations

import torch

from tests import train_ref as ref

U = 2.0 ** -24


def step_gradient(z, idx, inv, d_y, y_perm, router, alpha, p, seed, offset, counts, cu):
    """(gate part, balance part, bound) of the gradient of the scores z, for the loss whose
    gradient at the layer's output is d_y.

    bound: each part to 64 u of the magnitudes that it is the difference of (the balance
    part one more: alpha is rounded to fp32), u of the sum, and what the routing weights'
    gradient, itself to 64 u of its terms, brings in: w (dw_k - sum w dw) is linear in it.
    An expert that was not picked is given nothing for the gate part."""
    w = ref.weights(z.double().gather(1, idx.long()), router)
    _, dw, dw_size, _ = ref.combine_grad(d_y, y_perm, inv, w, p, seed, offset)
    gate, gate_size = ref.route_grad(z, idx, router, 0.0, dw, None, 1.0, None, cu)
    bal, bal_size = ref.route_grad(z, idx, router, alpha, None, counts, 1.0, None, cu)
    _, carried = ref.route_grad(z, idx, router, 0.0, 64 * U * dw_size, None, 1.0, None, cu)
    bound = 64 * U * gate_size + carried + 65 * U * bal_size + U * (gate + bal).abs()
    return gate, bal, bound


def weight_gradient(d_scores, x):
    """(d_scores^T x, bound): T products and their sum in fp32, in any order."""
    a, b = d_scores.double(), x.double()
    return a.t() @ b, (a.shape[0] + 1) * U * (a.abs().t() @ b.abs())
