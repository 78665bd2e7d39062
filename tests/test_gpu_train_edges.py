"""The router's training operators on the GPU where inputs are wrong or not finite:
expert ids outside the range, scores that are NaN or infinite.  Tolerances as derived in
tests/test_gpu_train.py."""
import pytest
import torch

from tests import train_ref as ref
from tests.test_gpu_train import (ROUTERS, U, _balance, _near, _route_backward, _scores,
                                  moe)  # noqa: F401  (moe is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("E,K", [(8, 2), (60, 6), (256, 8), (7, 5)])
@pytest.mark.parametrize("bal", [False, True])
def test_wrong_ids_take_no_part_in_the_gradient(moe, E, K, bal, router):  # noqa: F811
    """A slot whose id is outside [0, E) is in neither the softmax nor the sums of its token:
    the others' gradient is that of a token without it.  A token of such slots alone has the
    balance loss's part, or zeros."""
    T, alpha = 83, 0.3
    g, z, idx = _scores(T, E, K, 31)
    dw = torch.randn(T, K, generator=g)
    wild = torch.tensor([-1, E, 1 << 30, -(1 << 31), E + 1], dtype=torch.int64).int()
    wrong = torch.rand(T, K, generator=g) < 0.3
    wrong[5], wrong[6], wrong[T - 1] = True, False, True
    bad = torch.where(wrong, wild[torch.randint(0, 5, (T, K), generator=g)], idx)
    counts = torch.randint(0, 50, (1, E), generator=g, dtype=torch.int32) if bal else None
    got = _route_backward(moe, z, bad, router, alpha, dw, counts, 1.5 if bal else None)
    want, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    if bal:
        want, size = ref.route_grad(z, idx, router, alpha, None, counts, 1.5)
    for t in range(T):
        ok = ~wrong[t]
        if ok.any():
            a, b = ref.route_grad(z[t:t + 1], idx[t:t + 1, ok], router, alpha, dw[t:t + 1, ok])
            want[t] += a[0]
            size[t] += b[0]
    _near(got, want, 64 * U * size + U * want.abs())
    if not bal:
        assert (got[5] == 0).all() and (got[T - 1] == 0).all()


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("E,K", [(8, 2), (60, 6), (256, 8), (7, 5), (1000, 3)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_scores_that_are_not_finite_show(moe, E, K, what, router):  # noqa: F811
    """A NaN (or +inf) score of a token that takes part is not passed over: the token's
    gradient is NaN, and so are its sequence's mean probabilities and the loss.  Counts,
    the other tokens' gradients and the other sequences' means keep their bits."""
    T, alpha, cu = 300, 0.2, [0, 90, 200, 300]
    g, z, idx = _scores(T, E, K, 41)
    mask = torch.ones(T, dtype=torch.uint8)
    mask[7] = 0
    dw = torch.randn(T, K, generator=g)
    spoilt = z.clone()
    value = float(what)
    spoilt[120, idx[120, K - 1].long()] = value  # a picked expert's
    last = next(e for e in range(E) if e not in idx[133].tolist())
    spoilt[133, last] = value                    # one that was not picked
    spoilt[7, 0] = value                         # of a masked token
    hit = torch.zeros(T, dtype=torch.bool)
    hit[120] = hit[133] = True

    clean = _balance(moe, z, idx, router, alpha, mask, cu)
    counts, mean, loss, err = _balance(moe, spoilt, idx, router, alpha, mask, cu)
    assert err == 0 and torch.equal(counts, clean[0])
    assert torch.isnan(mean[1]).all() and torch.isnan(loss).all()
    assert torch.equal(mean[[0, 2]], clean[1][[0, 2]])

    for d, c in ((None, counts), (dw, counts)):
        want = _route_backward(moe, z, idx, router, alpha, d, c, None, mask, cu).cpu()
        got = _route_backward(moe, spoilt, idx, router, alpha, d, c, None, mask, cu).cpu()
        assert torch.isnan(got[hit]).all()
        assert torch.equal(got[~hit], want[~hit])
    # without the balance loss only the picked scores are read
    want = _route_backward(moe, z, idx, router, alpha, dw, None, None, mask, cu).cpu()
    got = _route_backward(moe, spoilt, idx, router, alpha, dw, None, None, mask, cu).cpu()
    assert torch.isnan(got[120][idx[120].long()]).all() and torch.isnan(got[120]).sum() == K
    hit[133] = False
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("router", ROUTERS)
def test_not_finite_in_one_block(moe, router):  # noqa: F811
    """The same where one block has every token."""
    T, E, K = 20, 8, 2
    _, z, idx = _scores(T, E, K, 42)
    z[11, 2] = float("nan")
    counts, mean, loss, err = _balance(moe, z, idx, router, 0.1)
    assert err == 0 and torch.isnan(mean).all() and torch.isnan(loss).all()
    assert counts.sum() == T * K


@pytest.mark.parametrize("router", ROUTERS)
@pytest.mark.parametrize("E,K", [(8, 2), (60, 6), (256, 8), (7, 5), (1000, 3)])
@pytest.mark.parametrize("d_loss", ["nan", "inf", "-inf"])
def test_masked_rows_are_zero_whatever_the_loss_gradient(moe, E, K, d_loss, router):  # noqa: F811
    """A loss scaled past fp32's range gives d_loss that is not finite: tokens that take part
    get NaN or infinities, masked ones and those outside every sequence zeros all the same."""
    T, cu = 300, [4, 90, 200, 290]
    g, z, idx = _scores(T, E, K, 43)
    mask = (torch.rand(T, generator=g) > 0.3).to(torch.uint8)
    dead = mask == 0
    dead[:4] = dead[290:] = True
    wild = z.clone()
    wild[mask == 0] = float("nan")
    counts, _, _, _ = _balance(moe, z, idx, router, 0.2, mask, cu)
    for dw in (None, torch.randn(T, K, generator=g)):
        got = _route_backward(moe, wild, idx, router, 0.2, dw, counts, float(d_loss), mask, cu).cpu()
        assert (got[dead] == 0).all()
        assert not torch.isfinite(got[~dead]).all(1).any()


@pytest.mark.parametrize("router", ROUTERS)
def test_masks_of_truth_values(moe, router):  # noqa: F811
    """token_mask as a comparison gives it (torch.bool) is the same mask as in bytes."""
    T, E, K = 200, 16, 3
    g, z, idx = _scores(T, E, K, 51)
    keep = torch.rand(T, generator=g) > 0.3
    dw = torch.randn(T, K, generator=g)
    a = _balance(moe, z, idx, router, 0.1, keep.to(torch.uint8))
    b = _balance(moe, z, idx, router, 0.1, keep)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    assert torch.equal(_route_backward(moe, z, idx, router, 0.1, dw, a[0], None, keep.to(torch.uint8)),
                       _route_backward(moe, z, idx, router, 0.1, dw, a[0], None, keep))
    with pytest.raises(ValueError, match="token_mask must be"):
        _balance(moe, z, idx, router, 0.1, keep.int())
