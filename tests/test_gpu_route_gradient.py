"""moe_route_backward where a score is close to one or to nothing, against the
gradients in 50 decimal digits.

Every value is a product of scores and of differences of gradients, none of
them a difference of two nearly equal sums:
  renormalized      scale q_j sum_i q_i (g_j - g_i)   (times 1 - s_j: sigmoid)
  plain softmax     scale p_e sum_i p_i (G_e - G_i)   over all experts
  plain sigmoid     scale g_j s_j (1 - s_j)
Tolerance: half a step of the output's type, and of the sum of absolute terms
2^-42.  A score takes an exponential of a difference of two logits (rounded:
2^-53 of at most 128, so 2^-46 of the value) and a few more steps of 2^-53;
gradients are taken against the largest score's, which is at least 1/64 of the
sum, so a difference to it is at most 64 times the sum of the absolute terms
and its roundings at most 2^-46 of that sum."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# subnormals lie 2^-149 apart in fp32 and 2^-133 in bf16 (2^-126 / 2^7), whose
# half step is 2^-134; fp32's whole step covers the rounding before bf16's
SMALL = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134 + 2.0 ** -149}


def exact(g, l, ids, scoring, renorm, scale):
    """(gradients, sums of absolute terms) as float64 [T, E]."""
    T, E = l.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    with localcontext() as c:
        c.prec = 50
        scale = Decimal(scale)
        for t in range(T):
            x = [Decimal(float(v)).exp() for v in l[t]]
            if scoring == "sigmoid":
                s = [v / (1 + v) for v in x]
                rest = [1 / (1 + v) for v in x]  # 1 - s
            else:
                z = sum(x)
                s, rest = [v / z for v in x], [Decimal(1)] * E
            at = [int(e) for e in ids[t]]
            gt = [Decimal(float(v)) for v in g[t]]
            d, a = [Decimal(0)] * E, [Decimal(0)] * E
            if renorm:
                total = sum(s[e] for e in at)
                q = [s[e] / total for e in at]
                for j, e in enumerate(at):
                    f = scale * q[j] * rest[e]
                    d[e] += f * sum(qi * (gt[j] - gi)
                                    for qi, gi in zip(q, gt))
                    a[e] += f * sum(qi * abs(gt[j] - gi)
                                    for qi, gi in zip(q, gt))
            elif scoring == "sigmoid":
                for j, e in enumerate(at):
                    d[e] += scale * gt[j] * s[e] * rest[e]
                    a[e] += abs(scale * gt[j] * s[e] * rest[e])
            else:
                G = [Decimal(0)] * E
                for j, e in enumerate(at):
                    G[e] += gt[j]
                for e in range(E):
                    d[e] = scale * s[e] * sum(p * (G[e] - v)
                                              for p, v in zip(s, G))
                    a[e] = scale * s[e] * sum(p * abs(G[e] - v)
                                              for p, v in zip(s, G))
            out[t] = [float(v) for v in d]
            size[t] = [float(v) for v in a]
    return out, size


def check(l, ids, g, scoring, renorm, scale, dtype=torch.float32):
    l = l.to(dtype)
    got = mxq.moe_route_backward(
        g.to(DEV), l.to(DEV), ids.to(DEV), scoring=scoring,
        renormalize=renorm, weight_scale=scale).cpu().double().numpy()
    want, size = exact(g.numpy(), l.double().numpy(), ids.numpy(), scoring,
                       renorm, scale)
    off = np.abs(got - want)
    lim = HALF[dtype] * 1.001 * np.abs(want) + 2.0 ** -42 * size + SMALL[dtype]
    assert (off <= lim).all(), (np.argwhere(~(off <= lim))[:4].tolist(),
                                got[~(off <= lim)][:4],
                                want[~(off <= lim)][:4])


def ids_of(rng, T, E, K):
    return torch.from_numpy(np.stack(
        [rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_saturated_sigmoid(dtype):
    """1 - s far below s: logits up to 85, where e^-l is a small fp32 value."""
    rng = np.random.default_rng(1)
    l = torch.linspace(-85, 85, 171).unsqueeze(1) + \
        torch.from_numpy(rng.uniform(0, 1, (171, 6))).float()
    g = torch.from_numpy(rng.standard_normal((171, 3))).float()
    say("saturated sigmoid", dtype)
    check(l, ids_of(rng, 171, 6, 3), g, "sigmoid", False, 1.5, dtype)


@pytest.mark.parametrize("K", [1, 2, 8])
def test_sigmoids_near_nothing(K):
    """Scores whose sum is so small that its reciprocal is beyond 64 bits:
    the weights, and their gradients, are of ordinary size."""
    rng = np.random.default_rng(2)
    l = torch.from_numpy(-709.7 + rng.uniform(0, 3, (40, 16))).float()
    l[:8] = -709.75
    l[8:16] = -600
    g = torch.from_numpy(rng.standard_normal((40, K))).float()
    g[0] = 1
    say("sigmoids near nothing", K)
    check(l, ids_of(rng, 40, 16, K), g, "sigmoid", True, 2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring,renorm", [("softmax", True),
                                            ("softmax", False),
                                            ("sigmoid", True)])
def test_one_score_far_above_the_others(scoring, renorm, dtype):
    """Its gradient is what the others leave of one; the others' hang on the
    difference to its gradient, which may be small or nothing."""
    rng = np.random.default_rng(3)
    T, E, K = 90, 12, 5
    l = torch.from_numpy(rng.standard_normal((T, E)) - 40).float()
    ids = ids_of(rng, T, E, K)
    top = rng.integers(0, K, T)
    for t in range(T):
        e = ids[t, top[t]] if t % 3 else E - 1  # chosen, or maybe not
        l[t, e] = -40 + t
    g = torch.from_numpy(rng.standard_normal((T, K))).float()
    g[::4] = g[::4, :1]                          # all equal
    g[1::4] = g[1::4, :1] * (1 + 2.0 ** -20 * torch.from_numpy(
        rng.standard_normal((len(g[1::4]), K))).float())
    say("one score far above", scoring, renorm, dtype)
    check(l, ids, g, scoring, renorm, 2.5, dtype)
