"""The bounds of the balance loss's sums: they agree with the other reference,
and a token left out of the sums breaks each of them (CPU)."""
import numpy as np
import pytest

import balance_bounds as bb
import fp8_mx_activation_amd as mxq
import mx_refs as mx


def batch(T, E, K, seed):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * 2 + 0.7 * rng.standard_normal(E)
    l = l.astype(np.float32).astype(np.float64)
    l[:, E // 3] = -np.inf
    return l, np.argsort(-l, 1)[:, :K].astype(np.int32)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_against_the_other_reference(scoring):
    l, ids = batch(200, 19, 3, 1)
    l[5] = -np.inf
    l[9, 4] = np.nan
    ids[7, 1] = -1
    off, lens = [3, 40, 40, 199], [30, 2, 200]
    a = mx.balance(l, ids, scoring, off, lens, 3)
    b = bb.forward(l, ids, scoring, off, lens, 3)
    for x, y in zip(a[:4], b[:4]):
        assert np.allclose(x, y, rtol=1e-13, atol=0)
    more = 1 + 1e-9  # the bounds' own rounding
    assert (b[5] <= more * (a[5] + mx.EPS * a[1])).all()
    assert (b[6] <= more * (a[4] + mx.EPS * a[3])).all()


@pytest.mark.parametrize("T,E,off", [(40, 16, None), (700, 24, None),
                                     (3000, 96, [0, 100, 2990]),
                                     (20000, 96, None)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_a_lost_token_shows(scoring, T, E, off):
    l, ids = batch(T, E, 4, T)
    S = 1 if off is None else len(off) - 1
    want = bb.forward(l, ids, scoring, off, None, S)
    for drop in (0, T // 2, T - 11 if off else T - 1):
        got = bb.forward(l, ids, scoring, off, None, S, drop)
        for what, i, e in (("loss", 0, 4), ("z", 1, 5), ("probs", 3, 6)):
            assert (np.abs(got[i] - want[i]) > 2 * want[e]).any(), (what, drop)


def test_which_sizes_take_two_launches():
    for E in (1, 16, 17, 32, 33, 64, 256, 257, 512, 513, 1024):
        most = 8 * 512 // bb.row_lanes(E)
        assert mxq.moe_balance_loss_workspace_bytes(most, E, 3) == 0
        assert mxq.moe_balance_loss_workspace_bytes(most + 1, E, 3) > 0
