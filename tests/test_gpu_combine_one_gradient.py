"""moe_combine_backward for one of its two gradients: the bytes are those of
the call for both, with y or the weights left out."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def problem(T, K, H, tg):
    """Tokens with none to all of K assignments here."""
    rng = np.random.default_rng(H)
    s = np.full((T, K), -1, np.int32)
    rows = rng.permutation(T * K)
    at = 0
    for t in range(T):
        here = rng.permutation(K)[:t % (K + 1)]
        s[t, here] = rows[at:at + len(here)]
        at += len(here)
    gen = torch.Generator().manual_seed(H)
    g = torch.randn((T, H), generator=gen).to(TYPES[tg]).to(DEV)
    y = torch.randn((T * K, H), generator=gen).bfloat16().to(DEV)
    w = torch.randn((T, K), generator=gen).to(DEV)
    return g, y, torch.from_numpy(s).to(DEV), w


@pytest.mark.parametrize("tg", ["bf16", "f32"])
@pytest.mark.parametrize("H", [8, 520, 1528, 7168, 32768])
def test_one_gradient(H, tg):
    T, K = 40, 9
    g, y, s, w = problem(T, K, H, tg)
    say("combine_backward, one gradient", H, tg)

    def rows():
        return torch.full((T * K, H), 7.0, dtype=torch.bfloat16, device=DEV)

    gy, gw = mxq.moe_combine_backward(g, y, s, w, grad_y=rows())
    only_y, none = mxq.moe_combine_backward(g, y, s, w, grad_y=rows(),
                                            need_grad_weights=False)
    assert none is None and torch.equal(only_y, gy)
    none, only_w = mxq.moe_combine_backward(g, y, s, w, need_grad_y=False)
    assert none is None and torch.equal(only_w, gw)
    # y is not read for the rows' gradient: nor are its values
    nan = torch.full_like(y, float("nan"))
    again, _ = mxq.moe_combine_backward(g, nan, s, w, grad_y=rows(),
                                        need_grad_weights=False)
    assert torch.equal(again, gy)
    # nor the weights for their own
    _, again = mxq.moe_combine_backward(g, y, s, torch.full_like(
        w, float("nan")), need_grad_y=False)
    assert torch.equal(again, gw)


def test_nothing_here():
    g = torch.ones((5, 64), device=DEV)
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    s = torch.full((5, 4), -1, dtype=torch.int32, device=DEV)
    w = torch.ones((5, 4), device=DEV)
    gy, gw = mxq.moe_combine_backward(g, none, s, w, need_grad_weights=False)
    assert gy.shape == (0, 64) and gw is None
    gy, gw = mxq.moe_combine_backward(g, none, s, w, need_grad_y=False)
    assert gy is None and (gw == 0).all()


def test_refusals():
    g, y, s, w = problem(4, 2, 64, "f32")
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y, s, w, need_grad_y=False,
                                 need_grad_weights=False)
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y, s, w, grad_y=torch.empty_like(y),
                                 need_grad_y=False)
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y, s, w, grad_weights=w.clone(),
                                 need_grad_weights=False)
