"""The norm and its backward pass at sizes that every form of their kernels takes more than once:
teams, warps and blocks that go from row to row, in place too, and at the ends of the range.

The statement (tests/norm_ref.py) runs on the GPU in 64 bits.  Tolerances, with u = 2^-24 (half a
step of fp32) and h = half a step of the rows' type:
  s        the fp32 sum rounded once: equal bits.
  y        a thread adds <= 72 squares, then 10 lane and warp steps: < 96 u of the mean, half of it
           in the root, the root 4 u, 4 roundings more: 64 u, and h of the rounded value.
  scales   as y: 64 u.
  codes    half a step of E4M3: 2^-4 of a normal value, 2^-10 scales of a small one, and the 64 u
           of y, of the scale and of the quotient.
  d_x      a difference of two parts, each with the errors of two such sums: 128 u of the parts'
           magnitudes, and h of the value.
  d_weight a chain of the rows of a team (at most T / 152, the grid being 152 blocks or more),
           <= 64 teams, <= 24 blocks of a strand, 5 lane steps, 64 for r and 8 for the terms'
           own roundings: 168 + T / 152, in u of the magnitudes.
An absolute 1e-37 covers values that fp32 holds as denormals.
"""
import pytest
import torch

from tests import norm_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 1e-37
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


def _rows(T, d, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    return g, (torch.randn(T, d, generator=g, device="cuda") * size).to(dt)


def _near(got, want, tol):
    assert torch.isfinite(got).all()
    over = ((got.double() - want).abs() - tol - TINY).max().item()
    assert over <= 0, (over, (got.double() - want).abs().max().item())


def _norm(moe, x, r, w, eps, want_s, want_y, want_codes):
    T, d = x.shape
    s = torch.full_like(x, 9) if want_s else None
    y = torch.full_like(x, 9) if want_y else None
    codes = torch.zeros(T, d, dtype=torch.uint8, device="cuda") if want_codes else None
    sc = torch.zeros(T, device="cuda") if want_codes else None
    moe.moe_rmsnorm(x, r, w, eps, s, y, codes, sc)
    return s, y, codes, sc


def _check(x, r, w, eps, out, dtype):
    s, y, codes, sc = out
    total = ref.add(x, r)
    yr = ref.norm(total, w, eps)
    if s is not None:
        assert torch.equal(s, total)
    if y is not None:
        _near(y, yr, (64 * U + HALF[dtype]) * yr.abs())
    if codes is not None:
        sr = ref.scales(yr)
        _near(sc, sr, 64 * U * sr)
        v = codes.view(torch.float8_e4m3fn).double() * sr[:, None]
        _near(v, yr, (2.0 ** -4 + 192 * U) * yr.abs() + 2.0 ** -10 * sr[:, None])


# Lanes of a warp a row (5 to 201 columns: more rows than a wave of blocks has, a last turn that is
# partly live); a warp a row, of two vectors a lane and four, rows that are no multiple of the eight
# of a block; a block a row.
FORWARD = [(90001, 5), (90001, 21), (90001, 24), (131071, 37), (100003, 40), (70001, 99), (70001, 100),
           (40001, 128), (20001, 200), (20001, 201), (20011, 333), (20003, 480), (3001, 777),
           (2501, 500), (2501, 1000), (1217, 1024), (1217, 4096)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", FORWARD)
def test_norm(moe, T, d, dtype):
    g, x = _rows(T, d, DT[dtype], 3 * T + d)
    r = (torch.randn(T, d, generator=g, device="cuda") * 2).to(DT[dtype])
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(DT[dtype])
    for res in (None, r):
        for want in ((True, True, True), (False, True, False), (False, False, True)):
            _check(x, res, w, 1e-6, _norm(moe, x, res, w, 1e-6, *want), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(131071, 37), (20011, 333), (3001, 777), (2501, 1000)])
def test_norm_in_place(moe, T, d, dtype):
    """s in the residual's place and y in x's, many rows a block: the bits of separate buffers."""
    g, x = _rows(T, d, DT[dtype], 1)
    r = torch.randn(T, d, generator=g, device="cuda").to(DT[dtype])
    w = torch.randn(d, generator=g, device="cuda").to(DT[dtype])
    s, y, _, _ = _norm(moe, x, r, w, 1e-5, True, True, False)
    x1, r1 = x.clone(), r.clone()
    moe.moe_rmsnorm(x1, r1, w, 1e-5, r1, x1, None, None)
    assert torch.equal(r1, s) and torch.equal(x1, y)


# At least four turns: lanes a row (5 to 201 columns), a ring a warp (333, 400; 200 and 201 of
# fp32), a ring a block with two, four and five vectors a thread (2048 to 16384), and straight from
# memory (fp32, 12289 and 16384); whole vectors and rows that start within them.
BACKWARD = [(131071, 5), (131071, 21), (131071, 24), (131071, 37), (100003, 40), (70001, 99),
            (70001, 100), (40001, 128), (40000, 200), (40000, 201),
            (20011, 333), (20011, 400), (3001, 777), (2501, 2048), (2501, 2049), (3001, 4096),
            (1501, 4099), (1501, 7168), (1501, 7169), (701, 9000), (701, 9001), (701, 12289),
            (701, 16381), (701, 16384)]


def _gradients(T, d, dtype, seed):
    g, s = _rows(T, d, DT[dtype], seed)
    dy, ds = (torch.randn(T, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    return dy, s, (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(DT[dtype]), ds


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", BACKWARD)
def test_backward(moe, T, d, dtype):
    dy, s, w, ds = _gradients(T, d, dtype, T + 7 * d)
    ws = moe.alloc_rmsnorm_workspace(T, d)
    for with_ds in (None, ds):
        dx = torch.full((T, d), 9.0, dtype=DT[dtype], device="cuda")
        dw = torch.full((d,), 9.0, device="cuda")
        moe.moe_rmsnorm_backward(dy, s, w, 1e-6, with_ds, dx, dw, ws)
        x_, xs, w_, wm = ref.grads(dy, s, w, 1e-6, with_ds)
        _near(dx, x_, 128 * U * xs + HALF[dtype] * x_.abs())
        _near(dw, w_, (168 + -(-T // 152)) * U * wm)
        dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
        moe.moe_rmsnorm_backward(dy, s, w, 1e-6, with_ds, dx2, None, None)
        moe.moe_rmsnorm_backward(dy, s, w, 1e-6, with_ds, None, dw2, ws)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(131071, 37), (40000, 200), (20011, 333), (2501, 2048), (2501, 2049),
                                 (1501, 7169), (701, 12289), (701, 16384), (701, 16381)])
def test_backward_in_place(moe, T, d, dtype):
    """d_x over each of the arrays that it is made of, rows ahead being fetched meanwhile."""
    dy, s, w, ds = _gradients(T, d, dtype, 8)
    ws = moe.alloc_rmsnorm_workspace(T, d)
    dx, dw = torch.empty_like(s), torch.empty(d, device="cuda")
    moe.moe_rmsnorm_backward(dy, s, w, 1e-6, ds, dx, dw, ws)
    for which in range(3):
        a = [dy.clone(), s.clone(), ds.clone()]
        dw2 = torch.empty_like(dw)
        moe.moe_rmsnorm_backward(a[0], a[1], w, 1e-6, a[2], a[which], dw2, ws)
        assert torch.equal(a[which], dx) and torch.equal(dw, dw2)
