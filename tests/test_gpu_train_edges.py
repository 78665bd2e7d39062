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
