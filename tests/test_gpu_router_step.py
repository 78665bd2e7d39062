"""The joined step of examples/train_router.py on the GPU, part by part, against 64 bits
from what its kernels read (tests/router_step.py; that its bounds tell mistakes from
rounding is tested on the CPU)."""
import pytest
import torch

from tests import router_step as step
from tests import train_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T,d,E,K,sequences", [(64, 128, 8, 2, 2), (301, 256, 24, 5, 3)])
def test_router_step_part_by_part(T, d, E, K, sequences):
    from examples import train_router as ex
    layer = ex.RouterTrainer(T, d, E, K, 128, sequences=sequences)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    target = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    w_g = (torch.randn(E, d, generator=g, device="cuda") * d ** -0.5).requires_grad_()
    seed, off = (int(v) for v in layer.rng)
    z = (x.float() @ w_g.t()).detach()
    layer.step(x, target, w_g)
    # the gradient at the output, by the step's own operations
    err = layer.y.float() - target.float()
    d_y = (err * (2.0 / err.numel())).bfloat16().cpu()

    z, idx, inv = z.cpu(), layer.topk_idx.cpu(), layer.inv_perm.cpu().view(T, K)
    y_perm, cu = layer.y_perm.cpu(), layer.seq_offsets.tolist()
    assert torch.equal(idx.sort(1).values, z.topk(K, dim=1).indices.int().sort(1).values)
    w = ref.weights(z.double().gather(1, idx.long()), "softmax")
    assert ((layer.topk_w.cpu().double() - w).abs() <= 64 * U * w).all()
    y, size = ref.combine(y_perm, inv, layer.topk_w.cpu(), None, x.cpu(), layer.p, seed, off)
    assert ((layer.y.cpu().double() - y).abs() <= (K + 6) * U * size + 2.0 ** -8 * y.abs()).all()
    counts, _, loss = ref.balance(z.double(), idx, "softmax", layer.alpha, None, cu)
    assert torch.equal(layer.counts.cpu().long(), counts)
    assert (layer.balance.cpu().double()[0] - loss).abs() <= 405 * U * loss  # alpha rounded too

    gate, bal, bound = step.step_gradient(z, idx, inv, d_y, y_perm, "softmax", layer.alpha, layer.p,
                                          seed, off, counts, cu)
    over = (layer.d_scores.cpu().double() - gate - bal).abs() - bound
    assert over.max().item() <= 0, over.max().item()
    want, most = step.weight_gradient(layer.d_scores.cpu(), x.cpu())
    assert ((w_g.grad.cpu().double() - want).abs() <= most).all()
