"""The references of the balance loss, of 4-bit floats and of their products
against facts that do not come from them (CPU)."""
import numpy as np
import pytest
import torch

import mx_refs as mx
import operator_refs as ref


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(scoring):
    rng = np.random.default_rng(3)
    T, E, S = 11, 7, 3
    l = rng.standard_normal((T, E)) * 2
    l[4, 2] = -np.inf
    ids = np.argsort(-l, 1)[:, :2]
    off, lens = [0, 4, 4, 10], [3, 0, 6]
    g, gz = rng.standard_normal(S), rng.standard_normal(S)
    counts = mx.balance(l, ids, scoring, off, lens, S)[2]
    out, _ = mx.balance_backward(g, gz, l, counts, scoring, off, lens, S)

    def total(l):
        loss, z, *_ = mx.balance(l, ids, scoring, off, lens, S)
        return (g * loss).sum() + (gz * z).sum()

    h = 1e-6
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert out[t, e] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            # central differences: h^2 of a third derivative, 2^-52 / h
            assert abs((total(a) - total(b)) / (2 * h) - out[t, e]) < 1e-8
    assert (out[[3, 10]] == 0).all()  # padding, and behind the last sequence


def test_balance_of_a_balanced_routing_is_one():
    T, E = 12, 4
    l = np.zeros((T, E))
    ids = np.arange(T)[:, None] % E
    for scoring in ("softmax", "sigmoid"):
        loss, z, counts, probs, *_ = mx.balance(l, ids, scoring)
        assert loss[0] == 1 and (counts == 3).all() and (probs == 0.25).all()
        assert abs(z[0] - np.log(4) ** 2) < 1e-15
    # all choices and shares on one expert: E
    l[:] = -np.inf
    l[:, 1] = 0.5
    assert mx.balance(l, np.ones((T, 1), int), "softmax")[0][0] == E


def test_codes_of_all_bf16_values():
    """Against bisection by the definition: halfway values go to the even
    code, anything above 5 to 6."""
    x = (torch.arange(65536, dtype=torch.int32) << 16).view(torch.float32)
    x = x[torch.isfinite(x)].double().numpy()
    want = np.zeros(x.shape, np.uint8)
    for i, h in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        want += (np.abs(x) >= h) if i % 2 else (np.abs(x) > h)
    want += 8 * np.signbit(x).astype(np.uint8)
    assert (mx.codes(x) == want).all()
    assert (mx.E2M1[mx.codes(mx.E2M1)] == mx.E2M1).all()


def test_exponents():
    x = np.zeros((6, 32))
    for i, v in enumerate((6.0, 6.1, 4.0, 3.0, 2.0 ** -140, 3e38)):
        x[i, i] = v
    assert mx.exponents(x, "no_clip")[:, 0].tolist() == \
        [0, 1, 0, -1, -127, 126]
    assert mx.exponents(x, "ocp_floor")[:, 0].tolist() == \
        [0, 0, 0, -1, -127, 125]
    # no clipping: the payload's largest is above 3 and at most 6
    rng = np.random.default_rng(1)
    x = rng.standard_normal((100, 64)) * np.exp(rng.standard_normal((100, 1)))
    e = mx.exponents(x, "no_clip").astype(float)
    top = np.abs(x).reshape(100, 2, 32).max(-1) / 2 ** e
    assert (top > 3).all() and (top <= 6).all()


def test_packing():
    c = np.arange(32, dtype=np.uint8)[None] % 16
    q = mx.pack(c)
    assert q[0, 0] == 0x10 and q[0, 7] == 0xFE
    assert (mx.unpack(q) == c).all()


def test_check_quantized_sees_mistakes():
    rng = np.random.default_rng(2)
    y = rng.standard_normal((4, 64))
    q, s = mx.quant(y)
    live, err = np.ones(4, bool), np.full(y.shape, 1e-9)
    mx.check_quantized(y, err, q, s, live)
    for k in range(8):
        bad = q.copy()
        bad[k % 4, k * 3] ^= 1 << k
        back = np.abs(mx.values(bad, s, "mxfp4") - mx.values(q, s, "mxfp4"))
        if back.max() == 0:
            continue
        with pytest.raises(AssertionError):
            mx.check_quantized(y, err, bad, s, live)
    with pytest.raises(AssertionError):
        mx.check_quantized(y, err, q, s + 1, live)


def test_products_of_quantized_rows():
    """Against torch's product of the decoded values."""
    rng = np.random.default_rng(4)
    q = rng.integers(0, 256, (5, 32), np.uint8)
    s = rng.integers(120, 130, (5, 2), np.uint8)
    w = rng.integers(0, 256, (2, 8, 32), np.uint8)
    ws = rng.integers(120, 130, (2, 8, 2), np.uint8)
    y, err = mx.expert_matmul(q, s, "mxfp4", w, ws, np.array([0, 3, 5]),
                              np.array([2, 2]), None, "none", None, 8)
    x = torch.from_numpy(mx.values(q, s, "mxfp4"))
    for e, rows in ((0, [0, 1]), (1, [3, 4])):
        m = torch.from_numpy(mx.values(w[e], ws[e], "mxfp4"))
        assert np.array_equal(y[rows], (x[rows] @ m.t()).numpy())
    assert np.isnan(y[2]).all() and (err[[0, 1, 3, 4]] > 0).all()
    assert ref.E4M3[0x38] == 1.0
