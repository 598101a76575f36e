"""More tokens than one launch holds (2^32 threads): every token's result is
that of the same token in a small call."""
import pytest
import torch

import fp8_mx_activation_amd as mxq
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

P = 1024  # tokens of the small call


def repeated(small, T):
    n = -(-T // P)
    return small.repeat((n,) + (1,) * (small.dim() - 1))[:T]


def same(big, small):
    """Every token's values, block by block."""
    whole = big.shape[0] // P * P
    assert (big[:whole].view(-1, *small.shape) == small).all()
    assert torch.equal(big[whole:], small[:big.shape[0] - whole])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route(scoring):
    T = (1 << 26) + 9  # four tokens to a block of 256 threads
    l = torch.randn((P, 2), generator=torch.Generator().manual_seed(1)) \
        .bfloat16().to(DEV)
    ids, w = mxq.moe_route(l, 1, scoring=scoring, renormalize=False)
    gw = torch.arange(P, device=DEV).float().view(P, 1)
    gl = mxq.moe_route_backward(gw, l, ids, scoring=scoring,
                                renormalize=False)
    say("route, many tokens", scoring, T)
    big = repeated(l, T)
    big_ids, big_w = mxq.moe_route(big, 1, scoring=scoring, renormalize=False)
    same(big_ids, ids)
    same(big_w, w)
    del big_w
    big_gl = mxq.moe_route_backward(repeated(gw, T), big, big_ids,
                                    scoring=scoring, renormalize=False)
    same(big_gl, gl)


def test_scatter_rows_backward():
    T = (1 << 26) + 9  # a token to a block of 64 threads
    rows = torch.randn((P, 8), device=DEV).bfloat16()
    s = torch.arange(P, dtype=torch.int32, device=DEV).view(P, 1)
    say("scatter_rows_backward, many tokens", T)
    same(mxq.moe_scatter_rows_backward(rows, repeated(s, T)),
         mxq.moe_scatter_rows_backward(rows, s))


def test_combine_backward():
    T = (1 << 23) + 9  # a token to a block of 512 threads
    y = torch.randn((P, 8), device=DEV).bfloat16()
    g = torch.randn((P, 8), device=DEV).bfloat16()
    w = torch.randn((P, 1), device=DEV)
    s = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1)
    gy, gw = mxq.moe_combine_backward(g, y, s[:P], w)
    say("combine_backward, many tokens", T)
    big_gy, big_gw = mxq.moe_combine_backward(repeated(g, T), repeated(y, T),
                                              s, repeated(w, T))
    same(big_gy, gy)
    same(big_gw, gw)
