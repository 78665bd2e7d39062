"""The norm in front of the experts on the GPU against its plain 64-bit statement
(tests/norm_ref.py), through the binding.

Tolerances, with u = 2^-24 (half a step of fp32) and h = eps / 2 of the rows' type:
  s        the fp32 sum rounded once: equal bits.
  y        a thread adds <= 72 squares, then 10 lane and warp steps: < 96 u of the mean,
           half of it in the root, the root 2 last places (4 u), 4 roundings more: 64 u, and h of
           the rounded value.
  scales   as y: 64 u.
  codes    half a step of E4M3: 2^-4 of a normal value, 2^-10 scales of a small one,
           and the 64 u of y and of the scale.
  d_x      a difference of two parts, each with the errors of two such sums: 128 u of the
           parts' magnitudes, u of the sum, h of the value.
  d_weight a chain of the rows of a team, <= 64 teams, <= 20 blocks of a strand, 5 lane
           steps: 128 + rows of a team, and 8 for the terms, in u of the magnitudes.
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
SIZES = [(1, 1), (3, 7), (1000, 3), (5, 8), (700, 64), (257, 100), (64, 256), (130, 520), (33, 1001),
         (40, 1032), (129, 2880), (19, 4099), (7, 7168), (500, 7168), (3, 8200), (2, 16384),
         (5, 16383), (9, 12289)]


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


def _rows(T, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(T, 1, generator=g))
    return g, (torch.randn(T, d, generator=g) * size).to(dt)


def _near(got, want, tol):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - tol - TINY
    assert over.max().item() <= 0, (over.max().item(), (got - want).abs().max().item())


def _check(moe, x, r, w, eps, want_s, want_y, want_codes, dtype, stream=None):
    T, d = x.shape
    xc, wc = x.cuda(), w.cuda()
    rc = None if r is None else r.cuda()
    s = torch.full_like(xc, 9) if want_s else None
    y = torch.full_like(xc, 9) if want_y else None
    codes = torch.zeros(T, d, dtype=torch.uint8, device="cuda") if want_codes else None
    sc = torch.zeros(T, device="cuda") if want_codes else None
    torch.cuda.synchronize()
    moe.moe_rmsnorm(xc, rc, wc, eps, s, y, codes, sc, stream)
    torch.cuda.synchronize()
    total = ref.add(x, r)
    yr = ref.norm(total, w, eps)
    if want_s:
        assert torch.equal(s.cpu(), total)
    if want_y:
        _near(y, yr, 64 * U * yr.abs() + HALF[dtype] * yr.abs())
    if want_codes:
        sr = ref.scales(yr)
        _near(sc, sr, 64 * U * sr)
        v = codes.view(torch.float8_e4m3fn).cpu().double() * sr[:, None]
        _near(v, yr, (2.0 ** -4 + 192 * U) * yr.abs() + 2.0 ** -10 * sr[:, None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES)
def test_norm(moe, T, d, dtype):
    g, x = _rows(T, d, DT[dtype], 3 * T + d)
    r = (torch.randn(T, d, generator=g) * 2).to(DT[dtype])
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype])
    for res in (None, r):
        for want in ((True, True, True), (False, True, False), (False, False, True)):
            _check(moe, x, res, w, 1e-6, *want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 7168, 1001])
def test_rows_of_zeros_and_of_infinities(moe, dtype, d):
    """A row of zeros gives zeros and scale 1; a row that is not finite shows and spoils no
    other row."""
    g, x = _rows(70, d, DT[dtype], d)
    w = torch.ones(d).to(DT[dtype])
    x[5] = 0
    _check(moe, x, None, w, 1e-6, True, True, True, dtype)
    xc = x.cuda()
    bad = x.clone()
    bad[7, d // 2], bad[8, 0], bad[69, d - 1] = float("nan"), float("inf"), float("-inf")
    out, clean = torch.empty_like(xc), torch.empty_like(xc)
    codes = [torch.empty(70, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.empty(70, device="cuda") for _ in range(2)]
    moe.moe_rmsnorm(xc, None, w.cuda(), 1e-6, None, clean, codes[0], sc[0])
    moe.moe_rmsnorm(bad.cuda(), None, w.cuda(), 1e-6, None, out, codes[1], sc[1])
    torch.cuda.synchronize()
    keep = torch.ones(70, dtype=torch.bool)
    keep[[7, 8, 69]] = False
    assert torch.equal(out.cpu()[keep], clean.cpu()[keep])
    assert torch.equal(codes[0].cpu()[keep], codes[1].cpu()[keep])
    assert torch.equal(sc[0].cpu()[keep], sc[1].cpu()[keep])
    assert torch.isnan(out.cpu()[7]).all() and torch.isnan(out.cpu()[8, 0])
    assert sc[0][5].item() == 1.0 and (codes[0][5] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 7168, 1001])
def test_rows_of_denormal_numbers(moe, dtype, d):
    """Their scale is 2^-126, their codes are finite and within half the least step (2^-10)
    of it, or half a step of the value."""
    x = (torch.randn(9, d, generator=torch.Generator().manual_seed(d)) * 1e-40).to(DT[dtype])
    x[3] = 0
    x[:, 1] = 0
    w = torch.ones(d).to(DT[dtype])
    codes = torch.zeros(9, d, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(9, device="cuda")
    moe.moe_rmsnorm(x.cuda(), None, w.cuda(), 1e-6, None, None, codes, sc)
    torch.cuda.synchronize()
    low = 2.0 ** -126
    want = torch.full((9,), low)
    want[3] = 1.0
    assert torch.equal(sc.cpu(), want)
    v = codes.view(torch.float8_e4m3fn).cpu().double() * low
    y = ref.norm(x, w, 1e-6)
    # 2^-149: the product's own rounding among denormal numbers, thrice
    assert ((v - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * low + 3 * 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(9, 7168), (300, 200), (11, 999)])
def test_in_place(moe, dtype, T, d):
    """s in the residual's or x's place, y in x's: the bits of separate buffers."""
    g, x = _rows(T, d, DT[dtype], 1)
    r = torch.randn(T, d, generator=g).to(DT[dtype]).cuda()
    x, w = x.cuda(), torch.randn(d, generator=g).to(DT[dtype]).cuda()
    s, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_rmsnorm(x, r, w, 1e-5, s, y, None, None)
    x1, r1 = x.clone(), r.clone()
    moe.moe_rmsnorm(x1, r1, w, 1e-5, r1, x1, None, None)
    assert torch.equal(r1, s) and torch.equal(x1, y)
    x2, y2 = x.clone(), torch.empty_like(x)
    moe.moe_rmsnorm(x2, r, w, 1e-5, x2, y2, None, None)
    assert torch.equal(x2, s) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES + [(4000, 24), (2500, 1024), (20000, 5)])
def test_backward(moe, T, d, dtype):
    g, s = _rows(T, d, DT[dtype], T + 7 * d)
    dy, ds = (torch.randn(T, d, generator=g).to(DT[dtype]) for _ in range(2))
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DT[dtype])
    ws = moe.alloc_rmsnorm_workspace(T, d)
    for with_ds in (None, ds):
        dx = torch.full((T, d), 9.0, dtype=DT[dtype], device="cuda")
        dw = torch.full((d,), 9.0, device="cuda")
        moe.moe_rmsnorm_backward(dy.cuda(), s.cuda(), w.cuda(), 1e-6,
                                 None if with_ds is None else with_ds.cuda(), dx, dw, ws)
        torch.cuda.synchronize()
        x_, xs, w_, wm = ref.grads(dy, s, w, 1e-6, with_ds)
        _near(dx, x_, 128 * U * xs + HALF[dtype] * x_.abs())
        chain = -(-T // 152)  # rows of a team: at most this, the grid being 152 blocks or more
        _near(dw, w_, (136 + chain) * U * wm)
        dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
        args = (dy.cuda(), s.cuda(), w.cuda(), 1e-6, None if with_ds is None else with_ds.cuda())
        moe.moe_rmsnorm_backward(*args, dx2, None, None)
        moe.moe_rmsnorm_backward(*args, None, dw2, ws)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,d", [(6, 40), (5, 33)])
def test_backward_against_differences(moe, T, d):
    """d_x and d_weight against differences of the forward call in fp32: a step of 2^-7 makes
    the differences' own error about 2^-14 of the second derivative plus 2^-24 / 2^-7 of the
    loss's terms; 4e-3 covers both for values around one."""
    g = torch.Generator().manual_seed(5)
    x, dy = torch.randn(T, d, generator=g), torch.randn(T, d, generator=g)
    w = 1 + 0.2 * torch.randn(d, generator=g)
    ws = moe.alloc_rmsnorm_workspace(T, d)
    dx, dw = torch.empty(T, d, device="cuda"), torch.empty(d, device="cuda")
    moe.moe_rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), 1e-6, None, dx, dw, ws)

    def loss(x, w):
        y = torch.empty(T, d, device="cuda")
        moe.moe_rmsnorm(x.cuda(), None, w.cuda(), 1e-6, None, y, None, None)
        return (y.cpu().double() * dy.double()).sum().item()

    step = 2.0 ** -7
    for t, c in ((0, 0), (T - 1, d - 1), (2, d // 2)):
        up, down = x.clone(), x.clone()
        up[t, c] += step
        down[t, c] -= step
        assert abs((loss(up, w) - loss(down, w)) / (2 * step) - dx[t, c].item()) < 4e-3
        up, down = w.clone(), w.clone()
        up[c] += step
        down[c] -= step
        assert abs((loss(x, up) - loss(x, down)) / (2 * step) - dw[c].item()) < 4e-3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_in_place(moe, dtype):
    T, d = 300, 1032
    g, s = _rows(T, d, DT[dtype], 8)
    dy, ds, w = (torch.randn(*n, generator=g).to(DT[dtype]).cuda() for n in ((T, d), (T, d), (d,)))
    s, ws = s.cuda(), moe.alloc_rmsnorm_workspace(T, d)
    dx, dw = torch.empty_like(s), torch.empty(d, device="cuda")
    moe.moe_rmsnorm_backward(dy, s, w, 1e-6, ds, dx, dw, ws)
    for which in range(3):
        a = [dy.clone(), s.clone(), ds.clone()]
        dw2 = torch.empty_like(dw)
        moe.moe_rmsnorm_backward(a[0], a[1], w, 1e-6, a[2], a[which], dw2, ws)
        assert torch.equal(a[which], dx) and torch.equal(dw, dw2)


def test_stream_and_graph(moe):
    """On a stream of the caller's, captured and replayed with other inputs."""
    T, d = 37, 2880
    g, x = _rows(T, d, torch.bfloat16, 4)
    x = x.cuda()
    r, w = torch.randn(T, d, device="cuda").bfloat16(), torch.randn(d, device="cuda").bfloat16()
    s, y, y2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = moe.alloc_rmsnorm_workspace(T, d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            moe.moe_rmsnorm(x, r, w, 1e-6, s, y, None, None)
            moe.moe_rmsnorm_backward(y, s, w, 1e-6, r, dx, dw, ws)
    x.copy_(torch.randn(T, d, device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    moe.moe_rmsnorm(x, r, w, 1e-6, None, y2, None, None)
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    moe.moe_rmsnorm_backward(y2, s, w, 1e-6, r, dx2, dw2, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_past_two_to_the_31_elements(moe):
    """Rows whose elements start past 2^31: the last rows are those of a small call."""
    d, T = 16384, (1 << 31) // 16384 + 3
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, d, device="cuda").bfloat16()
    x[-3:] = tail
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    want = torch.empty_like(tail)
    moe.moe_rmsnorm(tail, None, w, 1e-6, None, want, None, None)
    moe.moe_rmsnorm(x, None, w, 1e-6, None, x, None, None)
    torch.cuda.synchronize()
    assert torch.equal(x[-3:], want) and (x[:3] == 0).all()
