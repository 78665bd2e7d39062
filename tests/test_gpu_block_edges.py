"""Calls of the norm and of the layer for a few tokens at the edge of what they take."""
import pytest
import torch

from tests import norm_ref

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


U = 2.0 ** -24


def _rows_of_size(T, d, dtype, least, most, seed):
    """Rows of magnitudes between the two, of either sign, the first row all of the largest."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = least + (most - least) * torch.rand(T, d, generator=g, device="cuda", dtype=torch.float64)
    v[0] = most
    return g, (v * (1 - 2 * torch.randint(0, 2, (T, d), generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(40, 24), (9, 333), (9, 1000), (3, 7168), (3, 16384), (3, 12289)])
@pytest.mark.parametrize("end", ["large", "small"])
def test_rows_at_the_ends_of_the_range(moe, end, T, d, dtype):
    """Rows whose squares add up to nearly the largest fp32 number, and, without an eps, rows whose
    mean square is nearly the smallest normal one (some values so small that their squares are
    denormal: each is off by 2^-150, 2^-24 of the mean).  Tolerances as for ordinary rows: the
    squares' own u at most doubles, 64 u of y becomes 65, 128 of d_x 130, and d_weight's sum
    of three rows in teams adds u for each of <= 64 teams, 64 for r and 8 for the terms."""
    half = torch.finfo(dtype).eps / 2
    if end == "large":
        most = (0.98 * torch.finfo(torch.float32).max / d) ** 0.5  # a bf16 step up is 2^-8: 0.8 %
        g, x = _rows_of_size(T, d, dtype, most / 2, most, d)
    else:
        g, x = _rows_of_size(T, d, dtype, 1.5 * 2.0 ** -63, 3 * 2.0 ** -63, d)
        x[1:, ::7] *= 2.0 ** -7
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    y, sc = torch.empty_like(x), torch.empty(T, device="cuda")
    codes = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm(x, None, w, 0.0, None, y, codes, sc)
    want = norm_ref.norm(x, w, 0.0)
    assert ((y.double() - want).abs() <= (65 * U + half) * want.abs()).all()
    s = norm_ref.scales(want)
    assert ((sc.double() - s).abs() <= 65 * U * s).all()
    v = codes.view(torch.float8_e4m3fn).double() * s[:, None]
    assert ((v - want).abs() <= (2.0 ** -4 + 195 * U) * want.abs() + 2.0 ** -10 * s[:, None]).all()

    dy = torch.randn(T, d, generator=g, device="cuda").to(dtype)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    moe.moe_rmsnorm_backward(dy, x, w, 0.0, None, dx, dw, moe.alloc_rmsnorm_workspace(T, d))
    a, am, b, bm = norm_ref.grads(dy, x, w, 0.0)
    assert ((dx.double() - a).abs() <= 130 * U * am + half * a.abs() + 1e-37).all()
    assert ((dw.double() - b).abs() <= 140 * U * bm).all()
