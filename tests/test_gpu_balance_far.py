"""The log-sum-exp penalty's gradient where logits end fp32's range: the
factor 2 g / n times the log-sum-exp may pass it, the gradients of experts
without a share must not."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
from gpu_util import DEV, f32_to_dev, say

pytestmark = pytest.mark.gpu
MAX = float(np.finfo(np.float32).max)
INF, NAN = float("inf"), float("nan")

ROWS = [  # +inf counts as the largest finite value
    [INF, 0.0, -INF, NAN, 5.0, -MAX, 1e38],
    [INF, INF, -INF, 0.0, -7.0, NAN, -INF],   # 2 shares of a half
    [-MAX, -INF, NAN, -MAX, -INF, -INF, -INF],
    [1.0, -2.0, -INF, NAN, 0.5, -300.0, 3e4],
    [3e38, 3e38, 3e38, 3e38, -INF, NAN, 1.0]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [7, 8, 40, 200, 600])
@pytest.mark.parametrize("factor", [0.25, 1.5, 1000.0, -3.0])
def test_z_gradient_of_far_logits(factor, E, scoring, dtype):
    say("far logits", factor, E, scoring, dtype)
    rows = torch.full((len(ROWS), E), -INF)
    rows[:, :7] = torch.tensor(ROWS)
    rows = rows.to(dtype)
    n = len(ROWS)
    gz = np.array([factor * n / 2], np.float32)
    l = rows.double()
    dead = torch.isnan(l) | (l == -INF)
    l = torch.where(dead, torch.full_like(l, -INF), l.clamp(max=MAX))
    lse = torch.logsumexp(l, 1, keepdim=True)
    want = factor * (lse * torch.softmax(l, 1))
    add = torch.linspace(-2, 2, n * E).reshape(n, E).to(dtype)
    counts = torch.ones((1, E), dtype=torch.int32, device=DEV)
    for a in (None, add):
        for g in (None, f32_to_dev([1.0])):
            # equal counts: the loss has no gradient
            got = mxq.moe_balance_loss_backward(
                g, rows.to(DEV), None if g is None else counts,
                scoring=scoring, grad_z=f32_to_dev(gz),
                add=None if a is None else a.to(DEV)).cpu()
            left = torch.zeros_like(add) if a is None else a
            assert torch.equal(got[dead], left[dead])
            assert not torch.isnan(got).any()
            exact = want + left.double()
            # exponents up to 3e4: exp(x) of e^-3e4 is 0; the share, the
            # factor, the sum are off by 40 steps of fp32 at most; results
            # that the type does not hold are infinite
            lim = (40 * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16
                                      else 2.0 ** -24)) * exact.abs()
            top = torch.finfo(dtype).max
            sure = exact.abs() <= top * (1 - 2.0 ** -7)
            off = (got.double() - exact).abs()
            assert (off <= lim + 1e-37)[sure].all()
            over = exact.abs() >= top * (1 + 2.0 ** -7)
            assert torch.equal(got[over].double(),
                               torch.sign(exact[over]) * INF)
