"""The router's training operators on the GPU against their plain 64-bit
statement (tests/train_ref.py), through the binding.

Tolerances, with u = 2^-24 (half a step of fp32) and h = eps / 2 of the stored
type, derived from the arithmetic:
  counts            exact.
  probabilities     expf 2 steps, reciprocal 1, products 2, a sum over the
                    experts of at most 32 + 5 adds: < 64 u relative; the mean
                    adds a chain of < 336 adds (a lane's tokens, lanes, warps,
                    partial rows): 400 u.
  loss              the same relative error, one rounding more.
  d_logits          each part is f (a - dot): the error of f, of dot's <= 37 adds
                    and of the subtraction, each relative to f (|a| + sum p |a|):
                    64 u of that magnitude, and u of the sum.
  rows              K + 2 terms in fp32: (K + 6) u of their magnitudes, and one
                    rounding to the stored type, h of the value.
  d_topk_w          a thread adds <= 32 products, then 5 lane steps and <= 16
                    warps: 64 u of the magnitudes.
An absolute 1e-37 covers values that fp32 holds as denormals.
"""
import numpy as np
import pytest
import torch

from tests import train_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 1e-37
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


def _near(got, want, tol):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all()
    over = (got - want).abs() - tol - TINY
    assert over.max().item() <= 0, (over.max().item(), (got - want).abs().max().item())


def _cuda(t):
    return None if t is None else t.cuda()


def _scores(T, E, K, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E, generator=g) * scale + shift)
    return g, z, z.topk(K, dim=1).indices.int()


def _balance(moe, z, idx, router, alpha, mask=None, cu=None, stream=None):
    (T, E), K = z.shape, idx.shape[1]
    s = moe.make_shape(T, 64, E, K, 64, 0, "f32", router)
    n = 1 if cu is None else len(cu) - 1
    ws = moe.alloc_balance_workspace(s, n)
    counts = torch.full((n, E), -9, dtype=torch.int32, device="cuda")
    mean = torch.full((n, E), -9.0, device="cuda")
    loss = torch.full((1,), -9.0, device="cuda")
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    moe.moe_balance_loss(s, z.cuda(), idx.cuda(), _cuda(mask), cud, alpha, counts, mean, loss, ws,
                         stream)
    torch.cuda.synchronize()
    return counts, mean, loss, moe.moe_get_device_error(ws)


def _route_backward(moe, z, idx, router, alpha, dw, counts, d_loss, mask=None, cu=None):
    (T, E), K = z.shape, idx.shape[1]
    s = moe.make_shape(T, 64, E, K, 64, 0, "f32", router)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    out = torch.full((T, E), -9.0, device="cuda")
    moe.moe_route_backward(s, z.cuda(), idx.cuda(), _cuda(dw), _cuda(mask), cud, alpha,
                           _cuda(counts), None if d_loss is None else torch.tensor([d_loss]).cuda(),
                           out)
    torch.cuda.synchronize()
    return out


def _check_router(moe, z, idx, router, mask=None, cu=None, seed=0):
    """Loss, counts, means and every combination of gradients."""
    (T, E), K = z.shape, idx.shape[1]
    alpha = 0.25
    counts, mean, loss, err = _balance(moe, z, idx, router, alpha, mask, cu)
    assert err == 0
    wc, wm, wl = ref.balance(z.double(), idx, router, alpha, mask, cu)
    assert torch.equal(counts.cpu().long(), wc)
    _near(mean, wm, 400 * U * wm)
    _near(loss[0], wl, 404 * U * wl)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(seed)) * 0.01
    for gate, bal, d_loss in ((True, True, 1.5), (False, True, None), (True, False, None)):
        c = wc.int() if bal else None
        got = _route_backward(moe, z, idx, router, alpha, dw if gate else None, c, d_loss, mask, cu)
        want, size = ref.route_grad(z, idx, router, alpha, dw if gate else None, c,
                                    1.0 if d_loss is None else d_loss, mask, cu)
        _near(got, want, 64 * U * size + U * want.abs())


ROUTERS = ["softmax", "sigmoid"]
# experts below, at and above each way a row lies over the lanes; odd ones go scalar
EXPERTS = [(1, 1), (2, 1), (4, 4), (7, 3), (8, 2), (12, 12), (16, 5), (31, 31), (32, 32), (60, 6),
           (64, 8), (65, 2), (100, 32), (128, 1), (250, 9), (256, 8), (257, 8), (512, 4), (510, 3),
           (1000, 10), (1021, 32), (1024, 8)]


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("E,K", EXPERTS)
def test_router_over_expert_counts(moe, E, K, router):
    _, z, idx = _scores(77, E, K, E)
    _check_router(moe, z, idx, router)


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 127, 1024, 5003])
@pytest.mark.parametrize("E,K", [(8, 2), (60, 4), (7, 2)])
def test_router_over_token_counts(moe, T, E, K, router):
    _, z, idx = _scores(T, E, K, T)
    _check_router(moe, z, idx, router)


SEQS = {"ragged": [0, 5, 5, 6, 300, 301, 700], "gaps": [3, 40, 650], "all_empty": [9, 9, 9],
        "one_empty_first": [0, 0, 700], "single_tokens": list(range(0, 701)),
        "many_empty": [0] * 40 + [350] * 40 + [700] * 40, "one": [0, 700],
        "more_than_tokens": [i * 7 // 9 for i in range(901)],
        # as many offsets as a warp holds in registers, and one more
        "offsets_256": [min(700, 3 * i) for i in range(256)],
        "offsets_257": [min(700, 3 * i) for i in range(257)]}


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("name", sorted(SEQS))
@pytest.mark.parametrize("E,K", [(6, 5), (8, 2), (64, 6), (256, 8)])
def test_router_over_sequences(moe, name, E, K, router):
    _, z, idx = _scores(700, E, K, 5)
    _check_router(moe, z, idx, router, None, SEQS[name])


@pytest.mark.parametrize("T", [1, 17, 32])
def test_few_tokens_in_many_sequences(moe, T):
    _, z, idx = _scores(T, 6, 5, T)
    mask = (torch.arange(T) % 5 != 3).to(torch.uint8)
    _check_router(moe, z, idx, "sigmoid", mask, [i * T // 383 for i in range(384)])


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("kind", ["some", "none_left", "one_left", "whole_sequence"])
def test_router_with_masked_tokens(moe, kind, router):
    """Masked rows hold NaN, infinities and wild expert ids: nothing of them is used."""
    T, E, K = 300, 16, 3
    g, z, idx = _scores(T, E, K, 6)
    cu = [0, 100, 180, 300]
    mask = {"some": (torch.rand(T, generator=g) > 0.4), "none_left": torch.zeros(T, dtype=bool),
            "one_left": torch.arange(T) == 150,
            "whole_sequence": ~((torch.arange(T) >= 100) & (torch.arange(T) < 180))}[kind].to(torch.uint8)
    mask = mask * 255  # any non-zero byte counts
    dead = mask == 0
    wild, bad = z.clone(), idx.clone()
    wild[dead] = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38]).repeat(E // 4)
    bad[dead] = 1 << 30
    alpha, dw = 0.1, torch.randn(T, K, generator=g)
    counts, mean, loss, err = _balance(moe, wild, bad, router, alpha, mask, cu)
    assert err == 0
    wc, wm, wl = ref.balance(z.double(), idx, router, alpha, mask, cu)
    assert torch.equal(counts.cpu().long(), wc)
    _near(mean, wm, 400 * U * wm)
    _near(loss[0], wl, 404 * U * wl)
    got = _route_backward(moe, wild, bad, router, alpha, dw, wc.int(), 1.0, mask, cu)
    want, size = ref.route_grad(z, idx, router, alpha, dw, wc, 1.0, mask, cu)
    assert (got.cpu()[dead] == 0).all()
    _near(got, want, 64 * U * size + U * want.abs())


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("scale,shift", [(1, -200.0), (1, -80.0), (1, -65.0), (1, -55.0),
                                         (1, -45.0), (1, -40.0), (1, -20.0), (1, 80.0), (30, 0.0), (0, 0.0),
                                         (1e-30, 0.0), (50, -300.0)])
def test_router_with_far_scores(moe, scale, shift, router):
    """Scores where a sigmoid or an exponential under- or overflows on its own.  Tops
    that differ by rounding alone are drawn apart by the seed's values."""
    _, z, idx = _scores(65, 24, 4, 7, scale, shift)
    if router == "sigmoid" and shift < -100:
        # every weight underflows in fp32 as the definition's a / (sum + 1e-6) does; the loss stays
        counts, mean, loss, err = _balance(moe, z, idx, router, 0.2)
        wc, wm, wl = ref.balance(z.double(), idx, router, 0.2)
        assert torch.equal(counts.cpu().long(), wc)
        _near(mean, wm, 400 * U * wm)
        _near(loss[0], wl, 404 * U * wl)
        return
    _check_router(moe, z, idx, router)


@pytest.mark.parametrize("router", ROUTERS)
def test_router_with_forbidden_experts(moe, router):
    """-inf scores: probability and gradient 0; a row of them all gives zeros."""
    T, E, K = 40, 12, 2
    g, z, _ = _scores(T, E, K, 8)
    z[torch.rand(T, E, generator=g) < 0.4] = float("-inf")
    z[:, 5] = 0.1  # one at least is left
    z[:, 3] = 0.2
    idx = z.topk(K, dim=1).indices.int()
    _check_router(moe, z, idx, router)
    z[7] = float("-inf")
    counts, mean, loss, err = _balance(moe, z, idx, router, 0.2)
    wc, wm, wl = ref.balance(z.double(), idx, router, 0.2)
    assert err == 0 and torch.equal(counts.cpu().long(), wc)
    _near(mean, wm, 400 * U * wm)
    got = _route_backward(moe, z, idx, router, 0.2, None, wc.int(), None)
    assert (got.cpu()[7] == 0).all() and torch.isfinite(got).all()


@pytest.mark.parametrize("E", [16, 256, 7])
def test_repeated_picks_are_added(moe, E):
    """A token that names an expert twice (no top-K does): both shares count, the same bits
    each time."""
    T, K = 33, 4
    g, z, idx = _scores(T, E, K, 9)
    idx[::2, 3] = idx[::2, 0]
    idx[1::4, 1] = idx[1::4, 0]
    idx[1::4, 2] = idx[1::4, 0]
    dw = torch.randn(T, K, generator=g)
    first = _route_backward(moe, z, idx, "softmax", 0.1, dw, None, None)
    want, size = ref.route_grad(z, idx, "softmax", 0.1, dw, None)
    _near(first, want, 64 * U * size + U * want.abs())
    for _ in range(3):
        assert torch.equal(first, _route_backward(moe, z, idx, "softmax", 0.1, dw, None, None))


def test_wrong_ids_and_offsets_are_recorded(moe):
    """Ids outside [0, E) and offsets that do not ascend within [0, T] are reported
    through the workspace; the ids' slots are dropped from counts and gradient."""
    T, E, K = 50, 8, 2
    g, z, idx = _scores(T, E, K, 10)
    bad = idx.clone()
    bad[4, 1], bad[9, 0], bad[20, 1] = -1, E, 1 << 30
    counts, _, _, err = _balance(moe, z, bad, "softmax", 0.1)
    assert err == moe.MOE_ERR_BOUNDS
    ok = (bad >= 0) & (bad < E)
    assert torch.equal(counts.cpu()[0].long(), torch.bincount(bad[ok].long(), minlength=E))
    got = _route_backward(moe, z, bad, "softmax", 0.1, torch.ones(T, K), None, None)
    assert torch.isfinite(got).all()
    for cu in ([0, 30, 20, 50], [-5, 50], [0, 51], [0, 1 << 30], [40, 10]):
        assert _balance(moe, z, idx, "softmax", 0.1, None, cu)[3] == moe.MOE_ERR_BOUNDS
        assert torch.isfinite(_route_backward(moe, z, idx, "softmax", 0.1, None,
                                              torch.ones(len(cu) - 1, E, dtype=torch.int32), None,
                                              None, cu)).all()
    assert _balance(moe, z, idx, "softmax", 0.1, None, [0, 20, 50])[3] == 0


def test_balance_of_no_tokens(moe):
    s = moe.make_shape(0, 64, 8, 2, 64, 0, "f32")
    ws = moe.alloc_balance_workspace(s, 2)
    counts = torch.full((2, 8), 5, dtype=torch.int32, device="cuda")
    mean, loss = torch.ones(2, 8, device="cuda"), torch.ones(1, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    moe.moe_balance_loss(s, e, torch.empty(0, 2, dtype=torch.int32, device="cuda"), None,
                         torch.zeros(3, dtype=torch.int32, device="cuda"), 0.1, counts, mean, loss, ws)
    assert not counts.any() and not mean.any() and not loss.any()


def test_router_is_the_same_on_every_run_and_stream(moe):
    _, z, idx = _scores(6000, 256, 8, 12)
    cu = [0, 1, 900, 2500, 6000]
    a = _balance(moe, z, idx, "sigmoid", 0.1, None, cu)
    ga = _route_backward(moe, z, idx, "sigmoid", 0.1, torch.ones(6000, 8), a[0].cpu(), None, None, cu)
    side = torch.cuda.Stream()
    for st in (None, side):
        side.wait_stream(torch.cuda.current_stream())
        b = _balance(moe, z, idx, "sigmoid", 0.1, None, cu, st)
        for x, y in zip(a[:3], b[:3]):
            assert torch.equal(x, y)
        gb = _route_backward(moe, z, idx, "sigmoid", 0.1, torch.ones(6000, 8), a[0].cpu(), None,
                             None, cu)
        assert torch.equal(ga, gb)


@pytest.mark.parametrize("E", [1024, 1023])
def test_router_past_two_to_the_31_scores(moe, E):
    """Rows of scores and of their gradient that lie beyond 2^31 elements: all scores 0
    but the last three rows', which are a sequence of their own."""
    T, K = (1 << 21) + 4099, 2
    z = torch.zeros(T, E, device="cuda")
    idx = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(T, 1)
    _, last, picks = _scores(3, E, K, 21)
    z[-3:], idx[-3:] = last.cuda(), picks.cuda()
    cu = [0, T - 3, T]
    s = moe.make_shape(T, 64, E, K, 64, 0, "f32")
    ws = moe.alloc_balance_workspace(s, 2)
    counts = torch.empty(2, E, dtype=torch.int32, device="cuda")
    mean, loss, out = torch.empty(2, E, device="cuda"), torch.empty(1, device="cuda"), torch.empty_like(z)
    cud = torch.tensor(cu, dtype=torch.int32).cuda()
    moe.moe_balance_loss(s, z, idx, None, cud, 0.5, counts, mean, loss, ws)
    moe.moe_route_backward(s, z, idx, None, None, cud, 0.5, counts, None, out)
    assert moe.moe_get_device_error(ws) == 0
    wc, wm, _ = ref.balance(last.double(), picks, "softmax", 0.5)
    assert torch.equal(counts[1].cpu().long(), wc[0])
    _near(mean[1], wm[0], 400 * U * wm[0])
    assert counts[0].cpu().tolist()[:3] == [T - 3, T - 3, 0] and counts[0].sum() == 2 * (T - 3)
    # two million equal terms in a tree of chains of at most 7000 adds
    _near(mean[0], torch.full((E,), 1.0 / E, dtype=torch.float64), 7000 * U / E)
    want, size = ref.route_grad(last, picks, "softmax", 0.25, None, wc)  # one of two sequences
    _near(out[-3:], want, 64 * U * size + U * want.abs())
    # a row of equal scores: a_e - mean(a), over E, at the picks and beside them
    a = 0.25 * E * (T - 3) / (K * (T - 3.0) ** 2)
    row = torch.full((E,), -2 * a / E / E, dtype=torch.float64)
    row[:2] += a / E
    for r in (0, T // 2, T - 4):
        _near(out[r], row, 64 * U * (2 * a / E))


def test_router_in_a_graph(moe):
    """Loss and backward captured together follow their inputs at each replay."""
    T, E, K, n = 300, 64, 4, 3
    s = moe.make_shape(T, 64, E, K, 64, 0, "f32", "sigmoid")
    ws = moe.alloc_balance_workspace(s, n)
    cu = torch.tensor([0, 50, 120, 300], dtype=torch.int32).cuda()
    z, idx = torch.empty(T, E, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
    dw, out = torch.empty(T, K, device="cuda"), torch.empty(T, E, device="cuda")
    counts = torch.empty(n, E, dtype=torch.int32, device="cuda")
    mean, loss = torch.empty(n, E, device="cuda"), torch.empty(1, device="cuda")

    def calls():
        moe.moe_balance_loss(s, z, idx, None, cu, 0.1, counts, mean, loss, ws)
        moe.moe_route_backward(s, z, idx, dw, None, cu, 0.1, counts, loss, out)

    def fill(seed):
        g, zz, ii = _scores(T, E, K, seed)
        z.copy_(zz), idx.copy_(ii), dw.copy_(torch.randn(T, K, generator=g))

    fill(1)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (2, 3):
        fill(seed)
        graph.replay()
        got = [t.clone() for t in (counts, mean, loss, out)]
        calls()
        for a, b in zip(got, (counts, mean, loss, out)):
            assert torch.equal(a, b)
        want, _, wl = ref.balance(z.cpu().double(), idx.cpu(), "sigmoid", 0.1, None, cu.tolist())
        assert torch.equal(got[0].cpu().long(), want)
        _near(got[2][0], wl, 404 * U * wl)


def test_balance_of_the_library_s_own_routing(moe):
    """moe_route's scores, picks and weights into the loss: the counts are moe_permute's."""
    T, E, K = 500, 64, 4
    _, z, _ = _scores(T, E, K, 13)
    s = moe.make_shape(T, 64, E, K, 64, 0, "f32", "sigmoid")
    ws = moe.alloc_workspace(s)
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    zc = z.cuda()
    moe.moe_route(s, None, None, None, zc, None, idx, w, ws)
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    moe.moe_permute(s, idx, None, counts, off, None, None, None, ws)
    got = _balance(moe, z, idx.cpu(), "sigmoid", 0.1)
    assert torch.equal(got[0][0], counts)


# ---- dropout ----------------------------------------------------------------

def _rng(seed, offset):
    as_i64 = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([as_i64(seed), as_i64(offset)], dtype=torch.int64).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 5, 7, 8, 9, 63, 64, 1000, 4099, 300_001])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(moe, n, dtype, residual):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(DT[dtype])
    r = torch.randn(n, generator=g).to(DT[dtype]) if residual else None
    y = torch.full((n + 64,), 7.0, dtype=DT[dtype], device="cuda")
    seed, off = 0x9E3779B97F4A7C15, (5 << 40) + n
    moe.moe_dropout(x.cuda(), _cuda(r), 0.3, _rng(seed, off), y[:n])
    assert (y[n:] == 7.0).all()  # nothing beyond the end
    want = ref.dropout(x, r, 0.3, seed, off)
    size = x.double().abs() / 0.7 + (r.double().abs() if residual else 0)
    h = torch.finfo(DT[dtype]).eps / 2
    _near(y[:n], want, 4 * U * size + h * want.abs())
    keep, _ = ref.keep_and_scale((n,), 0.3, seed, off)
    got = y[:n].cpu()
    assert torch.equal(got[~keep], r[~keep] if residual else torch.zeros_like(got[~keep]))


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -16, 0.1, 0.5, 0.9, 1 - 2.0 ** -16, 1.0])
def test_dropout_mask_follows_p(moe, p):
    """The elements that stay are the generator's, for thresholds that cut its bits all over."""
    n = 20_000
    x = torch.ones(n, device="cuda")
    y = torch.empty_like(x)
    moe.moe_dropout(x, None, p, _rng(3, 4) if p * 65536 >= 0.5 else None, y)
    keep, scale = ref.keep_and_scale((n,), p, 3, 4)
    assert torch.equal(y.cpu() != 0, keep)
    _near(y, keep.double() * scale, 2 * U * scale)


def test_dropout_drops_what_is_not_finite(moe):
    x = torch.tensor([float("nan"), float("inf")], device="cuda").repeat(512)
    y = torch.empty_like(x)
    moe.moe_dropout(x, None, 0.5, _rng(1, 1), y)
    keep, _ = ref.keep_and_scale((1024,), 0.5, 1, 1)
    got = y.cpu()
    assert (got[~keep] == 0).all() and not torch.isfinite(got[keep]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_in_place(moe, dtype):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5001, generator=g).to(DT[dtype]).cuda()
    r = torch.randn(5001, generator=g).to(DT[dtype]).cuda()
    y = torch.empty_like(x)
    moe.moe_dropout(x, r, 0.2, _rng(8, 8), y)
    a, b = x.clone(), r.clone()
    moe.moe_dropout(a, r, 0.2, _rng(8, 8), a)
    moe.moe_dropout(x, b, 0.2, _rng(8, 8), b)
    assert torch.equal(a, y) and torch.equal(b, y)


def test_dropout_gradient_is_the_same_call(moe):
    """D is its own transpose: <D(x), g> = <x, D(g)>, exactly where both are sums of one term."""
    n = 4096
    x, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    moe.moe_dropout(x, None, 0.4, _rng(2, 6), y)
    moe.moe_dropout(g, None, 0.4, _rng(2, 6), dx)
    assert torch.equal(y != 0, dx != 0)
    # each product twice rounded on either side
    assert torch.allclose(y.double() * g.double(), x.double() * dx.double(), rtol=4 * U, atol=0)


def test_dropout_past_two_to_the_31_elements(moe):
    n = (1 << 31) + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    moe.moe_dropout(x, None, 0.5, _rng(5, 7), x)
    for a in (0, (1 << 31) - 100, n - 4099, n - 11):
        m = min(4099, n - a)
        keep = torch.from_numpy(ref.random16(np.arange(a, a + m, dtype=np.uint64), 5, 7) >= 32768)
        assert torch.equal(x[a:a + m].cpu(), keep.to(torch.bfloat16) * 2)


def test_dropout_graph_draws_new_masks(moe):
    """A captured call reads the generator's words at each replay."""
    x, rng = torch.ones(10_000, device="cuda"), _rng(1, 0)
    y = torch.empty_like(x)
    moe.moe_dropout(x, None, 0.5, rng, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_dropout(x, None, 0.5, rng, y)
        rng[1] += 1
    for off in range(3):
        graph.replay()
        keep, _ = ref.keep_and_scale((10_000,), 0.5, 1, off)
        assert torch.equal(y.cpu() != 0, keep)


# ---- combine ----------------------------------------------------------------

def _combine_inputs(T, K, d, dtype, seed, drop_slots=False):
    g = torch.Generator().manual_seed(seed)
    inv = torch.randperm(T * K, generator=g).int().view(T, K)
    if drop_slots:
        inv[torch.rand(T, K, generator=g) < 0.3] = -1
        inv.view(-1)[0] = T * K
    rnd = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])  # noqa: E731
    return dict(y_perm=rnd(T * K, d), inv=inv, w=torch.rand(T, K, generator=g), sh=rnd(T, d),
                res=rnd(T, d), d_y=rnd(T, d))


# widths around each way a row lies over threads; slots from one to the most
COMBINE = [(1, 1, 64), (3, 2, 64), (5, 32, 128), (7, 3, 256), (9, 1, 320), (4, 8, 2048),
           (3, 5, 2112), (6, 2, 4096), (2, 9, 4160), (5, 8, 7168), (2, 17, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,d", COMBINE)
@pytest.mark.parametrize("shared,residual,p", [(True, True, 0.2), (False, False, 0.2),
                                               (True, False, 0.0), (False, True, 1.0)])
def test_combine_dropout(moe, T, K, d, dtype, shared, residual, p):
    c = _combine_inputs(T, K, d, dtype, d + K, drop_slots=K == 3)
    s = moe.make_shape(T, d, max(K, 4), K, 64, 0, dtype)
    y = torch.empty(T, d, dtype=DT[dtype], device="cuda")
    sh, res = (c["sh"] if shared else None), (c["res"] if residual else None)
    moe.moe_combine_dropout(s, c["y_perm"].cuda(), c["inv"].cuda(), c["w"].cuda(), _cuda(sh),
                            _cuda(res), p, _rng(17, 3) if p else None, y)
    want, size = ref.combine(c["y_perm"], c["inv"], c["w"], sh, res, p, 17, 3)
    _near(y, want, (K + 6) * U * size + torch.finfo(DT[dtype]).eps / 2 * want.abs())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,d", COMBINE)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_combine_backward(moe, T, K, d, dtype, p):
    c = _combine_inputs(T, K, d, dtype, d + 7 * K, drop_slots=K == 3)
    s = moe.make_shape(T, d, max(K, 4), K, 64, 0, dtype)
    dev = {k: v.cuda() for k, v in c.items()}
    rng = _rng(21, 1 << 35) if p else None
    rows = torch.full((T * K, d), 7.0, dtype=DT[dtype], device="cuda")
    dw = torch.full((T, K), 7.0, device="cuda")
    dsh = torch.empty(T, d, dtype=DT[dtype], device="cuda")
    moe.moe_combine_backward(s, dev["d_y"], dev["y_perm"], dev["inv"], dev["w"], p, rng, rows, dw, dsh)
    wz, ww, size, wr = ref.combine_grad(c["d_y"], c["y_perm"], c["inv"], c["w"], p, 21, 1 << 35)
    h = torch.finfo(DT[dtype]).eps / 2
    _near(dw, ww, 64 * U * size)
    _near(dsh, wz, (2 * U + h) * wz.abs())
    named = torch.zeros(T * K, dtype=bool)
    ok = (c["inv"] >= 0) & (c["inv"] < T * K)
    named[c["inv"][ok].long()] = True
    _near(rows[named.cuda()], wr[named], (4 * U + h) * wr[named].abs())
    assert (rows[~named.cuda()] == 7.0).all()  # rows that no slot names stay

    # each output alone gives the same bits, and the rows may replace their source
    for which in range(3):
        r2, w2, s2 = torch.full_like(rows, 7.0), torch.empty_like(dw), torch.empty_like(dsh)
        moe.moe_combine_backward(s, dev["d_y"], dev["y_perm"] if which == 1 else None, dev["inv"],
                                 dev["w"] if which == 0 else None, p, rng,
                                 r2 if which == 0 else None, w2 if which == 1 else None,
                                 s2 if which == 2 else None)
        assert torch.equal((r2, w2, s2)[which], (rows, dw, dsh)[which])
    over, gy = dev["y_perm"].clone(), dev["d_y"].clone()
    w3 = torch.empty_like(dw)
    moe.moe_combine_backward(s, gy, over, dev["inv"], dev["w"], p, rng, over, w3, gy)
    assert torch.equal(w3, dw) and torch.equal(gy, dsh)
    assert torch.equal(over[named.cuda()], rows[named.cuda()])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 512])
def test_dropped_slots_have_no_gradient(moe, d, dtype):
    """inv_perm -1 gives d_topk_w 0 even where the output's gradient is not finite."""
    T, K = 5, 3
    c = _combine_inputs(T, K, d, dtype, 3)
    c["inv"][2] = -1
    c["inv"][4, 1] = T * K
    c["d_y"][2], c["d_y"][4] = float("inf"), float("nan")
    s = moe.make_shape(T, d, 4, K, 64, 0, dtype)
    dw = torch.full((T, K), 7.0, device="cuda")
    moe.moe_combine_backward(s, c["d_y"].cuda(), c["y_perm"].cuda(), c["inv"].cuda(), None, 0.0, None,
                             None, dw, None)
    got = dw.cpu()
    assert (got[2] == 0).all() and got[4, 1] == 0 and torch.isnan(got[4, 0])
    assert torch.isfinite(got[[0, 1, 3]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_without_dropout_is_moe_combine(moe, dtype):
    T, K, d = 33, 4, 512
    c = {k: v.cuda() for k, v in _combine_inputs(T, K, d, dtype, 1).items()}
    s = moe.make_shape(T, d, 8, K, 64, 0, dtype)
    a, b = torch.empty_like(c["sh"]), torch.empty_like(c["sh"])
    moe.moe_combine(s, c["y_perm"], c["inv"], c["w"], c["sh"], a)
    moe.moe_combine_dropout(s, c["y_perm"], c["inv"], c["w"], c["sh"], None, 0.0, None, b)
    assert torch.equal(a, b)


def test_combine_mask_is_the_plain_calls(moe):
    """The combine's dropout keeps what moe_dropout keeps, and its output may be the residual."""
    T, K, d = 19, 2, 192
    c = {k: v.cuda() for k, v in _combine_inputs(T, K, d, "f32", 2).items()}
    s = moe.make_shape(T, d, 8, K, 64, 0, "f32")
    plain, y, both = (torch.empty_like(c["sh"]) for _ in range(3))
    moe.moe_combine(s, c["y_perm"], c["inv"], c["w"], None, plain)
    moe.moe_dropout(plain, None, 0.3, _rng(4, 4), y)
    moe.moe_combine_dropout(s, c["y_perm"], c["inv"], c["w"], None, None, 0.3, _rng(4, 4), both)
    assert torch.equal(y, both)
    res = c["res"].clone()
    moe.moe_combine_dropout(s, c["y_perm"], c["inv"], c["w"], None, res, 0.3, _rng(4, 4), res)
    assert torch.equal(res, both + c["res"])
    again = c["sh"].clone()
    moe.moe_combine_dropout(s, c["y_perm"], c["inv"], c["w"], again, None, 0.3, _rng(4, 4), again)
    other = torch.empty_like(again)
    moe.moe_combine_dropout(s, c["y_perm"], c["inv"], c["w"], c["sh"], None, 0.3, _rng(4, 4), other)
    assert torch.equal(again, other)


def test_combine_past_two_to_the_31_elements(moe):
    """Rows of expert outputs that lie beyond 2^31 elements."""
    T, K, d = 20_000, 8, 16384
    n = T * K
    y_perm = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    y_perm[-1], y_perm[0] = 3.0, 5.0
    inv = torch.arange(n, dtype=torch.int32, device="cuda").view(T, K)
    w = torch.ones(T, K, device="cuda")
    s = moe.make_shape(T, d, 8, K, 64, 0, "bf16")
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_combine_dropout(s, y_perm, inv, w, None, None, 0.5, _rng(1, 2), y)
    keep = torch.from_numpy(ref.random16(
        np.arange((T - 1) * d, T * d, dtype=np.uint64), 1, 2) >= 32768)
    assert torch.equal(y[-1].cpu(), keep.to(torch.bfloat16) * 6)
    dw = torch.empty(T, K, device="cuda")
    moe.moe_combine_backward(s, torch.ones_like(y), y_perm, inv, w, 0.0, None, y_perm, dw, None)
    assert dw[-1, -1].item() == 3.0 * d and dw[0, 0].item() == 5.0 * d
    assert (y_perm[-1] == 1).all() and (y_perm[n // 2] == 1).all()


def test_strided_and_wrong_tensors_are_refused(moe):
    s = moe.make_shape(8, 64, 8, 2, 64, 0, "f32")
    wide = torch.zeros(8, 16, device="cuda")
    idx = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    out = torch.empty(8, 8, device="cuda")
    call = lambda z, i, o: moe.moe_route_backward(s, z, i, torch.zeros(8, 2, device="cuda"),  # noqa: E731
                                                  None, None, 0.1, None, None, o)
    with pytest.raises(ValueError, match="contiguous"):
        call(wide[:, :8], idx, out)
    with pytest.raises(ValueError, match="elements"):
        call(wide, idx, out)
    with pytest.raises(ValueError, match="int32"):
        call(out, idx.long(), out)
    with pytest.raises(moe.MoeError):  # rows go in 16-byte vectors
        call(torch.zeros(65, device="cuda")[1:], idx, out)


# ---- the operators together -------------------------------------------------

def test_router_step_gradient_is_the_losses(moe):
    """One step of the example: d_scores through the library's calls against
    differentiating the same step in 64 bits (experts' outputs as the library stored
    them).  bf16 enters twice: y's rounding (2^-8 of |y|) in the error, and d_y's."""
    from examples import train_router as ex
    T, d, E, K = 64, 128, 8, 2
    layer = ex.RouterTrainer(T, d, E, K, 128, sequences=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    target = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    w_g = (torch.randn(E, d, generator=g, device="cuda") * d ** -0.5).requires_grad_()
    off = int(layer.rng[1])
    scores = (x.float() @ w_g.t()).detach()
    layer.step(x, target, w_g)

    z = scores.cpu().double().requires_grad_()
    idx, cu = layer.topk_idx.cpu(), layer.seq_offsets.tolist()
    inv = layer.inv_perm.cpu().view(T, K)
    w = ref.weights(z.gather(1, idx.long()), "softmax")
    rows = layer.y_perm.cpu().double()[inv.long()]
    keep, scale = ref.keep_and_scale((T, d), layer.p, 0, off)
    y = x.cpu().double() + (w[:, :, None] * rows).sum(1) * keep * scale
    task = (y - target.cpu().double()).square().mean()
    total = task + ref.balance(z, idx, "softmax", layer.alpha, None, cu)[2]
    want, = torch.autograd.grad(total, z)
    # each element of err is off by 2^-8 |y|, d_y by another 2^-8 |d_y|; a score's
    # gradient sums d of them over w (1 - w) <= 1/4 of a difference of two rows
    off_y = 2.0 ** -8 * (y.detach().abs() + (y.detach() - target.cpu().double()).abs()) * 2 / y.numel()
    size = (off_y[:, None] * rows.abs().sum(1, keepdim=True) * scale).sum(2)
    got = layer.d_scores.cpu().double()
    assert ((got - want).abs() <= size + 64 * U * want.abs() + TINY).all()
    assert torch.allclose(w_g.grad.cpu().double(), want.t() @ x.cpu().double(),
                          atol=(size.max() * x.float().abs().max().item() * T).item())


def test_example_learns_and_balances(moe):
    """The example's run: the student nears the teacher (the loss falls by far more
    than its spread), and no expert is lost."""
    from examples import train_router as ex
    tasks, balances = ex.train(steps=60, T=1024, log=None)
    assert np.isfinite(tasks).all() and np.isfinite(balances).all()
    assert np.mean(tasks[-10:]) < 0.8 * np.mean(tasks[:5])
    assert balances[-1] < 0.05 * 2  # alpha times 2: even use is alpha times 1
