"""The layer for a few tokens where its work is cut in ways that narrow layers do not show: a long
K in one unit, eight tokens a warp of scores, parts that stay empty; and a captured decode step
against its calls one by one.  The 64-bit statement and its bound are tests/few_ref.py's."""
import pytest
import torch

from examples import decode_block
from tests import few_ref as ref
from tests.test_gpu_few import FORMATS, Layer, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


def _inputs(T, d, E, K, I, router, fmt, seed):  # noqa: E741
    """few_ref.inputs without a shared expert, made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    c = dict(T=T, d=d, E=E, K=K, I=I, Is=0, router=router, fmt=fmt)
    c["w_g"] = (rnd(E, d) / d ** 0.5).bfloat16()
    c["bias"] = 0.1 * rnd(E)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    for t in range(T):
        for _ in range(1000):
            x[t] = rnd(d)
            if ref.route(x[t:t + 1].double() @ c["w_g"].double().T, c["bias"], K, router)[2] > 1e-4:
                break
    c["x"], c["residual"] = x, rnd(T, d).bfloat16()
    for n, rows, cols in (("w_gate", I, d), ("w_up", I, d), ("w_down", d, I)):
        v = rnd(E, rows, cols) / cols ** 0.5
        if fmt == "bf16":
            c[n] = v.bfloat16()
            continue
        if fmt == "fp8":
            s = v.abs().amax(-1, keepdim=True) / 448
            c["s" + n[1:]] = s[..., 0].contiguous()
        else:
            v = v.view(E, rows // 128, 128, cols // 128, 128)
            s = v.abs().amax((-3, -1), keepdim=True) / 448
            c["s" + n[1:]] = s[..., 0, :, 0].contiguous()
        c[n] = (v / s).reshape(E, rows, cols).to(ref.FP8).view(torch.uint8)
    return c


def _check_here(moe, c):
    layer = Layer(moe, c, 255)
    y = layer()
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(layer.ws) == 0
    want, tol = ref.layer(c)
    assert torch.isfinite(y).all()
    over = ((y.double() - want).abs() - tol).max().item()
    assert over <= 0, (over, (y.double() - want).abs().max().item(), want.abs().max().item())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 3, 11])
def test_units_over_a_long_k(moe, fmt, T):
    """Enough tiles that K is not cut: with 8-bit weights 41 tiles a unit both ways, an odd number
    past two chunks of h's scales and past the 32 block scales that a warp holds."""
    _check_here(moe, _inputs(T, 5248, 12, 12, 5248, "softmax", fmt, T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [2, 16])
def test_parts_of_a_long_k(moe, fmt, T):
    """Down units of 20 and 16 tiles beside gate and up units of 41."""
    _check_here(moe, _inputs(T, 5248, 2, 2, 9728, "sigmoid", fmt, 50 + T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [13, 16])
def test_scores_of_eight_tokens_a_warp(moe, fmt, T):
    _check_here(moe, _inputs(T, 2048, 256, 2, 128, "sigmoid", fmt, T))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(2, 128, 2, 2, 128, 16384), (3, 256, 4, 2, 16384, 128),
                                   (1, 128, 3, 1, 128, 8192), (1, 256, 2, 1, 16384, 128),
                                   (9, 128, 3, 2, 16384, 256), (16, 128, 8, 3, 256, 16384)])
def test_parts_that_stay_empty(moe, fmt, shape):
    """K of the down products is cut for the wider of the routed and the shared expert: the
    narrower one's last parts have nothing to add."""
    _check(moe, ref.inputs(*shape, "softmax", fmt, sum(shape)))


def test_captured_steps_are_the_calls_one_by_one(moe):
    size = dict(T=3, d=256, E=8, K=2, inter=128, inter_shared=128)
    _, rows = decode_block.main(**size, layers=2, steps=3, seed=0)
    g = torch.Generator(device="cuda").manual_seed(0)
    blocks = [decode_block.Block(**size, g=g) for _ in range(2)]
    x = torch.randn(3, 256, generator=g, device="cuda").bfloat16()
    normed = torch.empty_like(x)
    for step in rows:
        x.copy_(torch.randn(3, 256, generator=g, device="cuda"))
        for block in blocks:
            block(x, normed)
        assert torch.equal(x, step)
