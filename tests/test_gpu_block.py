"""The parts of a sparse block run together: norm, layer and residual for a few tokens; the
norm's 8-bit rows in the W8A8 layer; the norm's backward pass behind the router's.  Each part
is held to its 64-bit statement on the values that its kernels read."""
import pytest
import torch

from examples import decode_block
from tests import few_ref, norm_ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    import sparse_expert_ffn_moe_gb300 as m
    return m


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "blocks"])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_norm_then_few_tokens(moe, fmt, T):
    """h = x + attention; n = norm(h); y = h + layer(n)."""
    from tests.test_gpu_few import Layer
    c = few_ref.inputs(T, 512, 16, 3, 384, 256, "sigmoid", fmt, 10 + T)
    g = torch.Generator().manual_seed(3)
    x, r = (torch.randn(T, 512, generator=g).bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(512, generator=g)).bfloat16()
    h, n = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    layer = Layer(moe, c)
    moe.moe_rmsnorm(x.cuda(), r.cuda(), w.cuda(), EPS, h, n, None, None)
    layer.g["residual"] = h
    y = layer(x=n)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(layer.ws) == 0
    assert torch.equal(h.cpu(), norm_ref.add(x, r))
    want = norm_ref.norm(h.cpu(), w, EPS)
    assert ((n.cpu().double() - want).abs() - (2.0 ** -8 + 64 * U) * want.abs()).max() <= 0
    # the statement asserts that the choice of experts is clear at these rows
    c.update(x=n.cpu(), residual=h.cpu())
    want, tol = few_ref.layer(c)
    assert ((y.cpu().double() - want).abs() - tol).max() <= 0


def _w8a8_statement(c, xq, sx):
    """The W8A8 layer in 64 bits from 8-bit rows, h quantised per row as its definition says."""
    x = xq.view(few_ref.FP8).double() * sx.double()[:, None]
    z = c["x"].double() @ c["w_g"].double().T
    idx, w, _ = few_ref.route(z, c["bias"], c["K"], c["router"])
    y = torch.zeros_like(x)
    for e in [None] + sorted(set(idx.flatten().tolist())):
        t = list(range(len(x))) if e is None else [i for i in range(len(x)) if e in idx[i].tolist()]
        pre = "ws_" if e is None else "w_"
        gate, up, down = (few_ref.matrix(c, pre + n, e) for n in ("gate", "up", "down"))
        h = torch.nn.functional.silu(x[t] @ gate.T) * (x[t] @ up.T)
        h = h.float().bfloat16().float()
        s = h.abs().amax(1, keepdim=True) / 448
        h = (h / s).to(few_ref.FP8).double() * s.double()
        wt = 1 if e is None else \
            torch.stack([w[i, idx[i].tolist().index(e)] for i in t])[:, None]
        y[t] += wt * (h @ down.T)
    return y


@pytest.mark.parametrize("fmt", ["fp8", "blocks"])
@pytest.mark.parametrize("T", [3, 150])
def test_norm_in_8_bits_then_w8a8(moe, fmt, T):
    """The norm's codes in place of the layer's own quantisation.  With the codes that the
    layer would make, its bits; with the norm's, the 64-bit layer on them (the bars of the
    W8A8 layer: 1e-2 relative, a code of h moves where its bf16 value straddles a border)."""
    c = few_ref.inputs(T, 512, 8, 2, 384, 256, "softmax", fmt, 20 + T, True, False)
    g = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    s = moe.make_shape(T, 512, 8, 2, 384, 256, "bf16", "softmax")
    ws, experts = moe.alloc_workspace(s), moe.make_fp8_experts(g)
    plain, codes = ((moe.moe_forward_w8a8, moe.moe_forward_w8a8_codes) if fmt == "fp8" else
                    (moe.moe_forward_w8a8_blocks, moe.moe_forward_w8a8_blocks_codes))
    x = g["x"]
    q, sx = torch.empty(T, 512, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_quantize_fp8_rows(x, q, sx)
    plain(s, x, g["w_g"], g["bias"], experts, a, ws)
    codes(s, x, q, sx, g["w_g"], g["bias"], experts, b, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    # the norm's codes of other rows than the router's
    w = torch.ones(512).bfloat16().cuda()
    moe.moe_rmsnorm(g["x"], None, w, EPS, None, None, q, sx)
    codes(s, x, q, sx, g["w_g"], g["bias"], experts, b, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_error(ws) == 0
    want = _w8a8_statement(c, q.cpu(), sx.cpu())
    assert (b.cpu().double() - want).norm() < 1e-2 * want.norm()


def test_codes_call_refuses_what_is_missing(moe):
    s = moe.make_shape(2, 128, 2, 1, 128, 0, "bf16")
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    q, sx = torch.zeros(2, 128, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda")
    w_g = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    for a, b in ((None, sx), (q, None), (q[:1], sx), (q, sx.double())):
        with pytest.raises(ValueError):
            moe.moe_forward_w8a8_codes(s, x, a, b, w_g, None, moe.make_fp8_experts({}), x, None)


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_norm_backward_behind_the_router(moe, router):
    """A balance loss's gradient through scores, products and norm to the residual stream and
    the norm's weight, against 64-bit autograd of the whole on the same bf16 values.  The
    products are the caller's; what they round (their result to bf16: 2^-8 of a row of d_n
    values) sets the bar: 2^-8 of the gradient's magnitudes and the norm's own 128 u."""
    T, d, E, K, alpha = 90, 200, 12, 2, 0.5
    g = torch.Generator().manual_seed(9)
    s_ = torch.randn(T, d, generator=g).bfloat16()
    w = (1 + 0.1 * torch.randn(d, generator=g)).bfloat16()
    w_g = (torch.randn(E, d, generator=g) / d ** 0.5).bfloat16()
    ds = torch.randn(T, d, generator=g).bfloat16()
    n = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_rmsnorm(s_.cuda(), None, w.cuda(), EPS, None, n, None, None)
    z = n.float() @ w_g.cuda().float().T
    idx = z.topk(K, 1).indices.int()
    shape = moe.make_shape(T, 64, E, K, 64, 0, "f32", router)
    counts = torch.empty(1, E, dtype=torch.int32, device="cuda")
    mean, loss = torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_balance_loss(shape, z, idx, None, None, alpha, counts, mean, loss,
                         moe.alloc_balance_workspace(shape))
    dz = torch.empty_like(z)
    moe.moe_route_backward(shape, z, idx, None, None, None, alpha, counts, None, dz)
    dn = (dz @ w_g.cuda().float()).bfloat16()
    dx, dw = torch.empty_like(n), torch.empty(d, device="cuda")
    moe.moe_rmsnorm_backward(dn, s_.cuda(), w.cuda(), EPS, ds.cuda(), dx, dw,
                             moe.alloc_rmsnorm_workspace(T, d))
    torch.cuda.synchronize()
    # each part on what it read, then the whole against autograd
    a, am, b, bm = norm_ref.grads(dn.cpu(), s_, w, EPS, ds)
    assert ((dx.cpu().double() - a).abs() - (128 * U * am + 2.0 ** -8 * a.abs())).max() <= 0
    assert ((dw.cpu().double() - b).abs() - 256 * U * bm).max() <= 0
    sd, wd = s_.double().requires_grad_(), w.double().requires_grad_()
    rows = norm_ref.norm(sd, wd, EPS)
    rows = rows + (n.cpu().double() - rows).detach()  # the bf16 rows, rounding passed through
    zz = rows @ w_g.double().T
    p = torch.softmax(zz, 1) if router == "softmax" else \
        torch.sigmoid(zz) / torch.sigmoid(zz).sum(1, keepdim=True)
    f = counts.cpu().double()[0] * E / (K * T)
    total = alpha * (f * p.mean(0)).sum() + (sd * ds.double()).sum()
    ga, gb = torch.autograd.grad(total, (sd, wd))
    _, am, _, bm = norm_ref.grads(dn.cpu(), s_, w, EPS)
    assert ((dx.cpu().double() - ga).abs() - (2.0 ** -8 * (am + ga.abs()) + 2.0 ** -12 * am)).max() <= 0
    assert ((dw.cpu().double() - gb).abs() - 2.0 ** -8 * bm * 1.1).max() <= 0


def test_decode_example_runs(moe):
    """The captured stack gives the bits of its calls one by one."""
    blocks, rows = decode_block.main(T=3, d=256, E=8, K=2, inter=128, inter_shared=128, layers=2,
                                     steps=3)
    assert torch.isfinite(rows.float()).all() and rows.shape == (3, 3, 256)
    g = torch.Generator(device="cuda").manual_seed(0)
    again, same = decode_block.main(T=3, d=256, E=8, K=2, inter=128, inter_shared=128, layers=2,
                                    steps=3)
    assert torch.equal(rows, same)
    x = torch.randn(3, 256, generator=g, device="cuda").bfloat16()
    y, normed = x.clone(), torch.empty_like(x)
    for block in blocks:
        block(y, normed)
    z = x.clone()
    for block in again:
        block(z, normed)
    assert torch.equal(y, z)
