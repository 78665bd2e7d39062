"""The bounds of tests/router_step.py on the CPU: rounding to fp32 passes them, and
every mistake of the kind that a joined step can hold does not."""
import pytest
import torch

from tests import router_step as step
from tests import train_ref as ref

T, D, E, K, P, ALPHA = 64, 128, 8, 2, 0.1, 0.05
CU = [0, 32, 64]


def _inputs(router):
    """A step's tensors at the sizes and magnitudes of the example's."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, D, generator=g).bfloat16()
    z = (x.float() @ torch.randn(D, E, generator=g)) * D ** -0.5
    idx = z.topk(K, dim=1).indices.int()
    order = torch.argsort(idx.reshape(-1).long(), stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * K)
    inv = inv.view(T, K).int()
    y_perm = (torch.randn(T * K, D, generator=g) * 0.35).bfloat16()
    y, _ = ref.combine(y_perm, inv, ref.weights(z.double().gather(1, idx.long()), router), None, x,
                       P, 7, 1)
    d_y = ((y.bfloat16().float() - torch.randn(T, D, generator=g)) * (2.0 / (T * D))).bfloat16()
    counts, _, _ = ref.balance(z.double(), idx, router, ALPHA, None, CU)
    parts = step.step_gradient(z, idx, inv, d_y, y_perm, router, ALPHA, P, 7, 1, counts, CU)
    return x, z, idx, inv, d_y, y_perm, counts, parts


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_parts_are_the_autograd_of_the_step(router):
    x, z, idx, inv, d_y, y_perm, _, (gate, bal, _) = _inputs(router)
    zz = z.double().requires_grad_()
    w = ref.weights(zz.gather(1, idx.long()), router)
    keep, scale = ref.keep_and_scale((T, D), P, 7, 1)
    y = (w[:, :, None] * y_perm.double()[inv.long()]).sum(1) * keep * scale
    total = (y * d_y.double()).sum() + ref.balance(zz, idx, router, ALPHA, None, CU)[2]
    want, = torch.autograd.grad(total, zz)
    assert torch.allclose(want, gate + bal, rtol=1e-12, atol=1e-18)


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_bounds_tell_mistakes_from_rounding(router):
    _, z, idx, inv, d_y, y_perm, counts, (gate, bal, bound) = _inputs(router)
    want = gate + bal

    def share(got):
        return ((got.double() - want).abs() > bound).double().mean().item()

    assert share(want.float()) == 0
    assert share(torch.zeros_like(want)) > 0.95
    assert share(gate) > 0.9 and share(gate + bal / 2) > 0.9 and share(gate + 1.01 * bal) > 0.9
    # what concerns the picked experts alone shows at most of them
    picked = torch.zeros(T, E, dtype=torch.bool).scatter_(1, idx.long(), True)

    def at_picks(got):
        return ((got.double() - want).abs() > bound)[picked].double().mean().item()

    assert at_picks(bal) > 0.9 and at_picks(bal + 0.99 * gate) > 0.9
    other, _, _ = step.step_gradient(z, idx, inv, d_y, y_perm, router, ALPHA, P, 7, 2, counts, CU)
    assert at_picks(other + bal) > 0.9  # the mask of another offset
    swapped, _, _ = step.step_gradient(z, idx, inv.flip(1), d_y, y_perm, router, ALPHA, P, 7, 1,
                                       counts, CU)
    assert at_picks(swapped + bal) > 0.9  # a token's rows in the other order


def test_weight_gradient_bound_is_tight():
    x, _, _, _, _, _, _, (gate, bal, _) = _inputs("softmax")
    d = (gate + bal).float()
    want, bound = step.weight_gradient(d, x)
    assert ((d.t() @ x.float()).double() - want).abs().le(bound).all()
    for wrong in (torch.zeros_like(want), want * 0.999, step.weight_gradient(gate.float(), x)[0]):
        assert ((wrong - want).abs() > bound).double().mean() > 0.9
