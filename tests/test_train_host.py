"""The router's training operators on the host: their 64-bit reference pinned
(published test vectors, differences), and the argument checks of the library's
entry points, which refuse bad calls before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

from tests import train_ref as ref


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import sparse_expert_ffn_moe_gb300 as m
    return m


# ---- the reference ----------------------------------------------------------

def test_philox_published_vectors():
    """The known answers published with the generator."""
    f = M = 0xFFFFFFFF
    assert ref.philox4x32_10([0] * 4, [0, 0]) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert ref.philox4x32_10([f] * 4, [M, M]) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert ref.philox4x32_10([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344],
                             [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


@pytest.mark.parametrize("seed,offset,first", [(0, 0, 0), (3, 5, 13), ((7 << 40) + 1, 9 << 33, 1 << 36)])
def test_random16_is_the_generators_halves(seed, offset, first):
    got = ref.random16(np.arange(first, first + 40, dtype=np.uint64), seed, offset)
    for n, i in enumerate(range(first, first + 40)):
        w = ref.philox4x32_10([i // 8 & ref.M32, i // 8 >> 32, offset & ref.M32, offset >> 32],
                              [seed & ref.M32, seed >> 32])
        assert got[n] == w[i % 8 // 2] >> 16 * (i % 2) & 0xFFFF


def test_dropout_keeps_the_expectation():
    """Of n elements a share p +- 5 sigma is dropped, and the mean stays."""
    n, p = 200_000, 0.3
    keep, scale = ref.keep_and_scale((n,), p, 11, 2)
    share = 1 - keep.double().mean().item()
    assert abs(share - p) < 5 * (p * (1 - p) / n) ** 0.5
    assert scale == 65536 / (65536 - round(p * 65536))


@pytest.mark.parametrize("router", ["softmax", "sigmoid"])
def test_reference_gradient_is_the_losses_difference(router):
    """route_grad against central differences of balance() and of the weights."""
    g = torch.Generator().manual_seed(1)
    T, E, K, alpha = 7, 5, 2, 0.3
    z = torch.randn(T, E, generator=g, dtype=torch.float64)
    idx = z.topk(K, dim=1).indices
    dw = torch.randn(T, K, generator=g, dtype=torch.float64)
    mask, cu = [1, 1, 0, 1, 1, 1, 1], [0, 3, 3, 6]
    counts, _, _ = ref.balance(z, idx, router, alpha, mask, cu)
    got, _ = ref.route_grad(z, idx, router, alpha, dw, counts, 1.5, mask, cu)

    def total(zz):
        part = [t for t in range(T) if mask[t] and t < cu[-1]]
        w = ref.weights(zz.gather(1, idx), router)
        return 1.5 * ref.balance(zz, idx, router, alpha, mask, cu)[2] + (w[part] * dw[part]).sum()

    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(z)
            d[t, e] = h
            # central differences: error ~ h^2 times a third derivative of order one
            assert abs((total(z + d) - total(z - d)) / (2 * h) - got[t, e]) < 1e-8


def test_reference_combine_gradient_is_the_difference():
    g = torch.Generator().manual_seed(2)
    T, K, d, p = 3, 2, 8, 0.25
    yp = torch.randn(T * K, d, generator=g, dtype=torch.float64)
    inv = torch.randperm(T * K, generator=g).view(T, K)
    inv[1, 1] = -1  # a dropped slot
    w = torch.rand(T, K, generator=g, dtype=torch.float64)
    dy = torch.randn(T, d, generator=g, dtype=torch.float64)
    _, dw, _, rows = ref.combine_grad(dy, yp, inv, w, p, 4, 9)
    f = lambda yy, ww: (ref.combine(yy, inv, ww, None, None, p, 4, 9)[0] * dy).sum()  # noqa: E731
    h = 1e-6
    for i in range(T * K):
        e = torch.zeros_like(yp)
        e[i, 3] = h
        assert abs((f(yp + e, w) - f(yp - e, w)) / (2 * h) - rows[i, 3]) < 1e-8
        e = torch.zeros_like(w)
        e[i // K, i % K] = h
        assert abs((f(yp, w + e) - f(yp, w - e)) / (2 * h) - dw[i // K, i % K]) < 1e-8


# ---- refusals ---------------------------------------------------------------

FAKE, ODD = 1 << 20, (1 << 20) + 2  # never dereferenced: the checks fail first
BIG = 1 << 40


def _call(moe, name, good, **kw):
    args = dict(good, **kw)
    assert set(args) == set(good), "unknown argument"
    return getattr(moe.library(), name)(*args.values())


def test_balance_loss_refusals(moe):
    s = moe.make_shape(4, 64, 8, 2, 64, 0, "f32")
    good = dict(s=ctypes.byref(s), logits=FAKE, idx=FAKE, mask=None, cu=FAKE, n=3, alpha=0.1,
                counts=FAKE, mean=FAKE, loss=FAKE, ws=FAKE, nws=BIG, st=None)
    bad = lambda **kw: _call(moe, "moe_balance_loss", good, **kw)  # noqa: E731
    for name in ("logits", "idx", "counts", "mean", "loss"):
        assert bad(**{name: None}) == moe.MOE_ERR_INVALID_ARG
        assert bad(**{name: ODD}) == moe.MOE_ERR_INVALID_ARG
    assert bad(logits=FAKE + 4) == moe.MOE_ERR_INVALID_ARG  # rows go in 16-byte vectors
    assert bad(cu=ODD) == moe.MOE_ERR_INVALID_ARG
    assert bad(cu=None) == moe.MOE_ERR_INVALID_ARG          # three sequences, no offsets
    assert bad(n=0) == moe.MOE_ERR_INVALID_ARG
    assert bad(n=-1) == moe.MOE_ERR_INVALID_ARG
    assert bad(n=(1 << 20) + 1) == moe.MOE_ERR_UNSUPPORTED
    assert bad(ws=None) == moe.MOE_ERR_WORKSPACE
    assert bad(ws=FAKE + 8) == moe.MOE_ERR_WORKSPACE
    need = moe.moe_balance_workspace_bytes(s, 3)
    assert need > 0 and bad(nws=need - 1) == moe.MOE_ERR_WORKSPACE
    k9 = moe.make_shape(4, 64, 8, 9, 64, 0, "f32")
    assert bad(s=ctypes.byref(k9)) == moe.MOE_ERR_INVALID_ARG
    assert bad(s=None) == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_balance_workspace_bytes(k9, 1) == 0
    assert moe.moe_balance_workspace_bytes(s, 0) == 0
    assert moe.moe_balance_workspace_bytes(s, (1 << 20) + 1) == 0


def test_route_backward_refusals(moe):
    s = moe.make_shape(4, 64, 8, 2, 64, 0, "f32")
    good = dict(s=ctypes.byref(s), logits=FAKE, idx=FAKE, dw=FAKE, mask=None, cu=None, n=1,
                alpha=0.1, counts=FAKE, d_loss=FAKE, out=2 * FAKE, st=None)
    bad = lambda **kw: _call(moe, "moe_route_backward", good, **kw)  # noqa: E731
    size = 4 * 8 * 4  # bytes of the [T][E] scores: the gradient may not lie over them
    for out in (FAKE, FAKE + size - 16, FAKE - size + 16):
        assert bad(out=out) == moe.MOE_ERR_INVALID_ARG
    for name in ("logits", "out"):
        for p in (None, ODD, FAKE + 4):
            assert bad(**{name: p}) == moe.MOE_ERR_INVALID_ARG
    assert bad(dw=None, counts=None) == moe.MOE_ERR_INVALID_ARG
    assert bad(idx=None) == moe.MOE_ERR_INVALID_ARG
    for name in ("idx", "dw", "counts", "d_loss"):
        assert bad(**{name: ODD}) == moe.MOE_ERR_INVALID_ARG
    assert bad(n=2) == moe.MOE_ERR_INVALID_ARG
    assert bad(s=None) == moe.MOE_ERR_INVALID_ARG
    empty = moe.make_shape(0, 64, 8, 2, 64, 0, "f32")
    assert bad(s=ctypes.byref(empty), logits=None, out=None) == moe.MOE_OK


def test_dropout_refusals(moe):
    good = dict(n=100, dtype=moe.MOE_BF16, x=FAKE, res=None, p=0.1, rng=FAKE, y=FAKE, st=None)
    bad = lambda **kw: _call(moe, "moe_dropout", good, **kw)  # noqa: E731
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert bad(p=p) == moe.MOE_ERR_INVALID_ARG
    assert bad(rng=None) == moe.MOE_ERR_INVALID_ARG
    assert bad(rng=FAKE + 4) == moe.MOE_ERR_INVALID_ARG
    assert bad(n=-1) == moe.MOE_ERR_INVALID_ARG
    assert bad(dtype=2) == moe.MOE_ERR_INVALID_ARG
    for name in ("x", "y"):
        assert bad(**{name: None}) == moe.MOE_ERR_INVALID_ARG
    for name in ("x", "y", "res"):
        assert bad(**{name: FAKE + 8}) == moe.MOE_ERR_INVALID_ARG
    assert bad(n=0, x=None, y=None) == moe.MOE_OK


@pytest.mark.parametrize("name", ["moe_combine_dropout", "moe_combine_backward"])
def test_combine_refusals(moe, name):
    s = moe.make_shape(4, 64, 8, 2, 64, 0, "bf16")
    if name == "moe_combine_dropout":
        good = dict(s=ctypes.byref(s), y_perm=FAKE, inv=FAKE, w=FAKE, sh=FAKE, res=FAKE, p=0.1,
                    rng=FAKE, y=FAKE, st=None)
        rows, must = ("y_perm", "sh", "res", "y"), ("y_perm", "inv", "w", "y")
    else:
        good = dict(s=ctypes.byref(s), d_y=FAKE, y_perm=FAKE, inv=FAKE, w=FAKE, p=0.1, rng=FAKE,
                    d_rows=FAKE, d_w=FAKE, d_sh=FAKE, st=None)
        rows, must = ("d_y", "y_perm", "d_rows", "d_sh"), ("d_y", "inv")
    bad = lambda **kw: _call(moe, name, good, **kw)  # noqa: E731
    for a in must:
        assert bad(**{a: None}) == moe.MOE_ERR_INVALID_ARG
    for a in rows:
        assert bad(**{a: FAKE + 8}) == moe.MOE_ERR_INVALID_ARG
    assert bad(inv=ODD) == moe.MOE_ERR_INVALID_ARG
    assert bad(w=ODD) == moe.MOE_ERR_INVALID_ARG
    assert bad(rng=None) == moe.MOE_ERR_INVALID_ARG
    assert bad(p=1.5) == moe.MOE_ERR_INVALID_ARG
    assert bad(s=None) == moe.MOE_ERR_INVALID_ARG
    odd_d = moe.make_shape(4, 100, 8, 2, 64, 0, "bf16")
    assert bad(s=ctypes.byref(odd_d)) == moe.MOE_ERR_UNSUPPORTED
    if name == "moe_combine_backward":
        assert bad(d_rows=None, d_w=None, d_sh=None) == moe.MOE_ERR_INVALID_ARG
        assert bad(y_perm=None) == moe.MOE_ERR_INVALID_ARG  # d_w reads it
        assert bad(w=None) == moe.MOE_ERR_INVALID_ARG       # d_rows reads it


def test_binding_refuses_host_and_strided_tensors(moe):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_dropout(x, None, 0.0, None, x, stream=0)
    s = moe.make_shape(4, 64, 8, 2, 64, 0, "f32")
    with pytest.raises(ValueError, match="missing"):
        moe.moe_balance_loss(s, None, None, None, None, 0.1, None, None, None, None, stream=0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32])
def test_dropout_refuses_other_types(moe, dtype):
    x = torch.zeros(4, 8, dtype=dtype)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        moe.moe_dropout(x, None, 0.0, None, x, stream=0)


@pytest.mark.parametrize("name", ["moe_dropout", "moe_combine_dropout", "moe_combine_backward"])
def test_generator_is_asked_for_wherever_something_is_drawn(moe, name):
    """The threshold is 65536 p + 1/2 rounded down, in double: it is 1 from the largest
    double below 2^-17 on (the sum rounds to 1), and there the generator's words are
    read.  Asked of calls of no elements, which read nothing."""
    s = moe.make_shape(0, 64, 8, 2, 64, 0, "bf16")
    good = {"moe_dropout": dict(n=0, dtype=moe.MOE_BF16, x=None, res=None, p=0.0, rng=None, y=None,
                                st=None),
            "moe_combine_dropout": dict(s=ctypes.byref(s), y_perm=None, inv=None, w=None, sh=None,
                                        res=None, p=0.0, rng=None, y=None, st=None),
            "moe_combine_backward": dict(s=ctypes.byref(s), d_y=None, y_perm=None, inv=None, w=None,
                                         p=0.0, rng=None, d_rows=None, d_w=None, d_sh=None,
                                         st=None)}[name]
    edge = np.nextafter(2.0 ** -17, 0.0)
    for p in (0.0, 5e-324, 2.0 ** -18, np.nextafter(edge, 0.0), edge, 2.0 ** -17, 2.0 ** -16, 0.5, 1.0):
        draws = int(float(p) * 65536 + 0.5) > 0
        assert _call(moe, name, good, p=float(p)) == (moe.MOE_ERR_INVALID_ARG if draws else moe.MOE_OK)
        assert _call(moe, name, good, p=float(p), rng=FAKE) == moe.MOE_OK
