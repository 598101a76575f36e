"""moe_route and moe_route_backward against the 64-bit reference.

Ids must be equal.  The kernel's weights are 64-bit numbers rounded once to
fp32: half a step, 2^-24 relative, and nothing else above 2^-50.  Gradients
are rounded once to the logits' type (2^-24 or 2^-8, half a step); in a row of
cancelling terms the 64-bit steps before that are off by less than 2^-48 of
the largest term."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import operator_refs as ref
from gpu_util import DEV, assert_equal, host, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def logits_of(rng, T, E, dtype, spread=2.0):
    return torch.from_numpy(
        (spread * rng.standard_normal((T, E))).astype(np.float32)).to(
            TYPES[dtype])


def as64(t):
    return t.double().numpy()


def check(rng, l, K, dtype, what, **kw):
    say("route", what, tuple(l.shape), K, dtype, kw)
    bias = kw.get("bias")
    ids, w = mxq.moe_route(
        l.to(DEV), K, scoring=kw.get("scoring", "softmax"),
        bias=None if bias is None else torch.from_numpy(bias).to(DEV),
        num_groups=kw.get("groups", 1), top_groups=kw.get("top_groups", 1),
        renormalize=kw.get("renorm", True), weight_scale=kw.get("scale", 1.0))
    rid, rw = ref.route(as64(l), K, **kw)
    assert_equal(host(ids), rid, what + " ids")
    np.testing.assert_allclose(host(w).astype(np.float64), rw, rtol=2.0 ** -24
                               * 1.001, atol=2.0 ** -149, err_msg=what)
    return ids, w


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (3, 7, 7),
                                   (300, 60, 4), (17, 64, 6), (5, 65, 64),
                                   (33, 160, 6), (9, 257, 8), (257, 512, 10),
                                   (2, 1000, 64), (4, 1024, 1)])
def test_sizes(T, E, K, scoring, dtype):
    rng = np.random.default_rng(T * 1000 + E)
    l = logits_of(rng, T, E, dtype)
    check(rng, l, K, dtype, "plain", scoring=scoring)
    check(rng, l, K, dtype, "biased", scoring=scoring, renorm=False,
          scale=2.5,
          bias=(0.3 * rng.standard_normal(E)).astype(np.float32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,g,K", [(256, 8, 4, 8), (64, 64, 9, 9),
                                     (12, 4, 2, 6), (60, 3, 1, 5),
                                     (8, 2, 2, 8), (513, 27, 5, 20)])
def test_groups(E, G, g, K, scoring, dtype):
    rng = np.random.default_rng(E + G)
    l = logits_of(rng, 70, E, dtype)
    check(rng, l, K, dtype, "groups", scoring=scoring, groups=G,
          top_groups=g)
    check(rng, l, K, dtype, "groups, biased", scoring=scoring, groups=G,
          top_groups=g,
          bias=(0.3 * rng.standard_normal(E)).astype(np.float32))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_ties_and_odd_values(scoring, groups, top_groups):
    """Equal logits, masked experts (-inf, NaN, the type's lowest value),
    +inf, rows with nothing to choose, signed zeros."""
    rng = np.random.default_rng(5)
    E, K = 32, 6
    low = np.finfo(np.float32).min
    rows = [np.zeros(E), np.full(E, -0.0), np.full(E, -np.inf),
            np.full(E, np.nan), np.full(E, low), np.full(E, np.inf)]
    r = rng.standard_normal((12, E))
    r[0, ::2] = -np.inf
    r[1, 5:] = -np.inf
    r[2, 1:] = np.nan
    r[3, 3] = np.inf
    r[4, [3, 9]] = np.inf
    r[5, 8:] = low
    r[6] = np.round(r[6])
    r[7] = np.round(r[7])
    r[8, 8:16] = -np.inf
    r[9] *= 30
    r[10, :31] = -np.inf
    r[11, ::3] = -0.0
    l = torch.from_numpy(np.concatenate([np.stack(rows), r]).astype(
        np.float32))
    for renorm in (True, False):
        for bias in (None, np.where(np.arange(E) % 5 == 0, 0.25, 0).astype(
                np.float32)):
            check(rng, l, K, "f32", "odd values", scoring=scoring,
                  groups=groups, top_groups=top_groups, renorm=renorm,
                  bias=bias)
    # a bias that takes experts out
    bias = np.zeros(E, np.float32)
    bias[:30] = -np.inf
    bias[30] = np.nan
    check(rng, l, K, "f32", "bias masks", scoring=scoring, bias=bias)


def test_near_ties_go_by_64_bits():
    """Choice values that differ by less than fp32 can hold."""
    E = 64
    l = np.full((8, E), 3.0, np.float32)
    for t in range(8):
        l[t, 40 + t] = np.nextafter(np.float32(3.0), np.float32(4.0))
    bias = np.full(E, 4.0, np.float32)
    for scoring in ("softmax", "sigmoid"):
        ids, _ = check(np.random.default_rng(0), torch.from_numpy(l), 3,
                       "f32", "near ties", scoring=scoring, bias=bias)
        assert host(ids)[:, 0].tolist() == [40 + t for t in range(8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,g,K", [(256, 8, 4, 8), (256, 1, 1, 8),
                                     (96, 6, 2, 9), (1024, 16, 3, 5),
                                     (40, 40, 7, 7)])
def test_values_close_together(E, G, g, K, scoring, dtype):
    """Choice values, group sums and cut-offs that 32 bits cannot tell apart
    among others that they can, with and without a bias; saturated scores.

    A 64-bit value takes an exponential (one unit, 2^-52 of it), a sum, a
    quotient and the bias's sum (2^-53 each), a softmax's sum over the row
    1024 positive terms: 2^-42 of the value at most, two of them in a group's
    value.  What differs by less may go either way."""
    rng = np.random.default_rng(E + G)
    T = 96
    spread = 10.0 ** rng.uniform(-9, 0, (T, 1))
    centre = rng.choice([0.0, 0.0, 1.5, -3.0, 12.0, 20.0, 40.0, -720.0],
                        (T, 1))
    l = centre + spread * rng.standard_normal((T, E))
    l[:16] = 1e-8 * rng.integers(-3, 4, (16, E))
    l[16:24, ::3] = -np.inf
    l = torch.from_numpy(l.astype(np.float32)).to(TYPES[dtype])
    ties = np.where(rng.random(E) < 0.5, 0.25, -1.0)
    for bias in (None, ties, 2.0 ** -23 * rng.integers(0, 9, E),
                 rng.standard_normal(E), 30 * rng.standard_normal(E)):
        b = None if bias is None else bias.astype(np.float32)
        say("route close", E, G, g, K, scoring, dtype, b is None)
        ids, w = mxq.moe_route(
            l.to(DEV), K, scoring=scoring,
            bias=None if b is None else torch.from_numpy(b).to(DEV),
            num_groups=G, top_groups=g)
        ids, w = host(ids), host(w)
        L = ref.clean_logits(as64(l))
        for t in range(T):
            s = ref.scores(L[t], scoring)
            c = s + (0 if b is None else b.astype(np.float64))
            tol = 2.0 ** -40 * max(1.0, np.abs(c).max())
            live = L[t] > -np.inf
            c = np.where(live, c, -np.inf)
            two = -np.sort(-c.reshape(G, -1), axis=1)[:, :2]
            value = np.where(two > -np.inf, two, 0).sum(1)
            value[two[:, 0] == -np.inf] = -np.inf
            group = np.arange(E) // (E // G)
            better = (value[None] > value[:, None] + tol).sum(1)
            at_least = (value[None] >= value[:, None] - tol).sum(1) - 1
            may = live & (better[group] < g)       # in a group that may be kept
            must = live & (at_least[group] < g)    # in one that is kept
            got = ids[t][ids[t] >= 0]
            assert len(set(got.tolist())) == len(got) and may[got].all()
            assert (ids[t][len(got):] == -1).all()
            assert len(got) == K or must.sum() <= len(got)
            assert (c[got][:-1] >= c[got][1:] - tol).all()
            rest = must.copy()
            rest[got] = False
            if len(got):
                assert not (c[rest] > c[got].min() + tol).any(), t
            if b is None and G == 1 and scoring == "softmax":
                assert (L[t][got][:-1] >= L[t][got][1:]).all()
            p = s[got] / s[got].sum() if s[got].sum() > 0 else 0 * s[got]
            np.testing.assert_allclose(w[t][:len(got)], p, rtol=2.0 ** -23,
                                       atol=2.0 ** -149)


def test_strided_logits_and_given_outputs():
    rng = np.random.default_rng(9)
    for dtype, pad in (("f32", 3), ("bf16", 1), ("f32", 4), ("bf16", 8)):
        big = logits_of(rng, 40, 100 + pad, dtype).to(DEV)
        l = big[:, 1:101]
        ids = torch.full((40, 8), 77, dtype=torch.int32, device=DEV)
        w = torch.full((40, 8), 7.0, device=DEV)
        mxq.moe_route(l, 8, ids=ids, weights=w)
        rid, rw = ref.route(as64(l.cpu()), 8)
        assert_equal(host(ids), rid, "strided ids")
        np.testing.assert_allclose(host(w), rw, rtol=2.0 ** -24 * 1.001)
        # the gradient of a strided view into a strided view
        g = torch.randn((40, 8), device=DEV)
        out = torch.full((40, 100 + pad), 5.0, dtype=l.dtype, device=DEV)
        mxq.moe_route_backward(g, l, ids, grad_logits=out[:, 1:101])
        want = ref.route_backward(host(g), as64(l.cpu()), rid, "softmax",
                                  True, 1.0)
        close(out[:, 1:101], want, dtype, g)
        assert (out[:, 0] == 5).all() and (out[:, 101:] == 5).all()


def close(got, want, dtype, g, scale=1.0):
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    terms = scale * np.abs(host(g)).max()
    np.testing.assert_allclose(
        got.cpu().double().numpy(), want, rtol=half * 1.001,
        atol=max(terms * 2.0 ** -48, 2.0 ** -134))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (3, 7, 7),
                                   (300, 60, 4), (5, 65, 64), (9, 257, 8),
                                   (2, 1000, 33)])
def test_backward(T, E, K, renorm, scoring, dtype):
    rng = np.random.default_rng(E)
    l = logits_of(rng, T, E, dtype)
    l[0, 0] = -np.inf if E > 1 else 0.5
    ids, _ = ref.route(as64(l), K, scoring=scoring, renorm=renorm)
    g = torch.randn((T, K), generator=torch.Generator().manual_seed(E))
    say("route_backward", T, E, K, renorm, scoring, dtype)
    got = mxq.moe_route_backward(
        g.to(DEV), l.to(DEV), torch.from_numpy(ids).to(DEV),
        scoring=scoring, renormalize=renorm, weight_scale=1.5)
    want = ref.route_backward(g.numpy(), as64(l), ids, scoring, renorm, 1.5)
    close(got, want, dtype, g, 1.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(renorm, scoring):
    """The reference's gradient is the slope of the reference's weights, and
    the kernel's is the reference's."""
    rng = np.random.default_rng(3)
    l = logits_of(rng, 6, 20, "f32", 1.0)
    ids, _ = ref.route(as64(l), 5, scoring=scoring, renorm=renorm)
    g = rng.standard_normal((6, 5)).astype(np.float32)

    def loss(l64):
        total = np.zeros(6)
        for t in range(6):
            p = ref.scores(l64[t], scoring)[ids[t]]
            w = p / p.sum() if renorm else p
            total[t] = (2.0 * w * g[t]).sum()
        return total

    base = as64(l)
    h = 1e-5
    slope = np.zeros((6, 20))
    for e in range(20):
        up, dn = base.copy(), base.copy()
        up[:, e] += h
        dn[:, e] -= h
        slope[:, e] = (loss(up) - loss(dn)) / (2 * h)
    want = ref.route_backward(g, base, ids, scoring, renorm, 2.0)
    # central differences: error h^2/6 of the third derivative (at most about
    # ten times the gradients' size here) plus 2^-52 * |loss| / h
    np.testing.assert_allclose(slope, want, atol=1e-8)
    got = mxq.moe_route_backward(
        torch.from_numpy(g).to(DEV), l.to(DEV), torch.from_numpy(ids).to(DEV),
        scoring=scoring, renormalize=renorm, weight_scale=2.0)
    close(got, want, "f32", torch.from_numpy(g), 2.0)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_missing_and_repeated_ids(renorm, scoring):
    rng = np.random.default_rng(4)
    l = logits_of(rng, 5, 40, "f32")
    ids = np.array([[-1, -1, -1, -1], [3, 3, 3, 3], [0, -1, 39, 40],
                    [5, 5, 1 << 30, -(1 << 30)], [7, 8, 9, 10]], np.int32)
    g = rng.standard_normal((5, 4)).astype(np.float32)
    got = mxq.moe_route_backward(
        torch.from_numpy(g).to(DEV), l.to(DEV), torch.from_numpy(ids).to(DEV),
        scoring=scoring, renormalize=renorm)
    want = ref.route_backward(g, as64(l), ids, scoring, renorm, 1.0)
    # a repeated id adds its fp32 terms: one more rounding for each
    np.testing.assert_allclose(got.cpu().double().numpy(), want,
                               rtol=2.0 ** -21,
                               atol=2.0 ** -23 * np.abs(g).max())


def test_route_refusals():
    l = torch.zeros((4, 16), device=DEV)
    with pytest.raises(mxq.MxqError):
        mxq.moe_route(l, 17)
    with pytest.raises(mxq.MxqError):
        mxq.moe_route(l, 4, num_groups=3)
    with pytest.raises(KeyError):
        mxq.moe_route(l, 4, scoring="max")
    with pytest.raises(TypeError):
        mxq.moe_route(l.half(), 4)
    with pytest.raises(ValueError):
        mxq.moe_route(l, 4, bias=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        mxq.moe_route(l, 4, bias=torch.zeros(16))
    with pytest.raises(ValueError):
        mxq.moe_route(l, 4, ids=torch.zeros((4, 4), device=DEV))
    with pytest.raises(ValueError):
        mxq.moe_route(l.t(), 4)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        mxq.moe_route_backward(torch.zeros((4, 3), device=DEV), l, ids)
    with pytest.raises(TypeError):
        mxq.moe_route_backward(torch.zeros((4, 2), device=DEV), l, ids,
                               grad_logits=l.bfloat16())
    i, w = mxq.moe_route(l[:0], 4)
    assert tuple(i.shape) == (0, 4) and tuple(w.shape) == (0, 4)


@pytest.mark.parametrize("E", [1, 5, 64, 200, 256, 1000, 1024])
def test_every_bf16_value(E):
    """All bf16 bit patterns as logits, NaNs and infinities among them, each
    beside others drawn at random and its own repetition."""
    rng = np.random.default_rng(E)
    bits = rng.permutation(65536).astype(np.uint16)
    pad = (-len(bits)) % E
    bits = np.concatenate([bits, bits[:pad]]).reshape(-1, E)
    bits = bits[rng.permutation(len(bits))[:512]]
    bits[:, E // 2:] = bits[:, :E - E // 2]
    l = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16)
    check(rng, l, min(E, 9), "bf16", "bf16 values")
    check(rng, l, min(E, 9), "bf16", "bf16 values", renorm=False)
