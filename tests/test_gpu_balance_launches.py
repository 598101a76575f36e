"""moe_balance_loss in two launches, every width of rows, against sums that
leave no room for a lost token, and its gradient; and on both sides of the most
tokens that one launch takes."""
import numpy as np
import pytest
import torch

import balance_bounds as bb
import fp8_mx_activation_amd as mxq
import mx_refs as mx
from gpu_util import assert_equal, f32_to_dev, host, i32_to_dev, say
from test_gpu_balance import HALF, problem

pytestmark = pytest.mark.gpu


def check(l, ids, scoring, offsets=None, lens=None, gradient=True):
    S = 1 if offsets is None else len(offsets) - 1
    kw = dict(scoring=scoring,
              seq_offsets=None if offsets is None else i32_to_dev(offsets),
              seq_lens=None if lens is None else i32_to_dev(lens))
    L = l.double().cpu().numpy()
    loss, z, counts, probs, lerr, zerr, perr = bb.forward(
        L, host(ids), scoring, offsets, lens, S)
    for with_z in (True, False):
        r = mxq.moe_balance_loss(l, ids, z_loss=with_z, **kw)
        assert_equal(host(r["counts"]), counts.astype(np.int32), "counts")
        assert (np.abs(host(r["probs"]) - probs) <= perr).all()
        assert (np.abs(host(r["loss"]) - loss) <= lerr).all()
        assert ("z_loss" in r) == with_z
        if with_z:
            assert (np.abs(host(r["z_loss"]) - z) <= zerr).all()
    if not gradient:
        return
    T = L.shape[0]
    rng = np.random.default_rng(T)
    g = rng.standard_normal(S).astype(np.float32) * T
    for gz in (None, rng.standard_normal(S).astype(np.float32) * T):
        out = mxq.moe_balance_loss_backward(
            f32_to_dev(g), l, r["counts"],
            grad_z=None if gz is None else f32_to_dev(gz), **kw)
        want, err = mx.balance_backward(g, gz, L, counts, scoring, offsets,
                                        lens, S)
        off = np.abs(out.double().cpu().numpy() - want)
        assert (off <= err + HALF[out.dtype] * (np.abs(want) + err)).all()


# one width of rows after the other, E % 4 == 0 and not, just above and some
# way above the most tokens of one launch
SIZES = [(1025, 16), (1100, 6), (513, 32), (700, 21), (257, 40), (520, 64),
         (270, 100), (520, 130), (257, 192), (300, 195), (520, 200),
         (600, 256), (129, 512), (300, 400), (131, 263), (65, 1024),
         (200, 600), (70, 513)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E", SIZES)
def test_two_launches(T, E, dtype, scoring):
    assert mxq.moe_balance_loss_workspace_bytes(T, E, 1) > 0
    say("balance in two launches", T, E, dtype, scoring)
    l, ids = problem(T + E, T, E, min(E, 5), dtype, dead=1)
    check(l, ids, scoring)
    cuts = [2, 3, 3, 20, T // 2, T - 7, T]
    check(l, ids, scoring, cuts, [1, 0, 9, T, T // 4, 7], gradient=False)


@pytest.mark.parametrize("E", [16, 32, 64, 128, 192, 256, 512, 1024])
def test_the_most_tokens_of_one_launch(E):
    T = 8 * 512 // bb.row_lanes(E)
    assert mxq.moe_balance_loss_workspace_bytes(T, E, 1) == 0
    say("balance in one launch", T, E)
    l, ids = problem(E, T, E, 4)
    check(l, ids, "softmax", gradient=False)
    check(l, ids, "sigmoid", [0, 1, T - 1], gradient=False)


@pytest.mark.parametrize("T,E,dtype", [(40000, 96, torch.bfloat16),
                                       (8192, 256, torch.float32),
                                       (30011, 17, torch.float32),
                                       (3000, 1000, torch.bfloat16)])
def test_many_tokens(T, E, dtype):
    """Several rows a lane in every block."""
    l, ids = problem(T, T, E, 6, dtype)
    for scoring in ("softmax", "sigmoid"):
        say("balance of many tokens", T, E, dtype, scoring)
        check(l, ids, scoring, gradient=False)
        check(l, ids, scoring, [0, 100, T // 2, T // 2 + 1, T - 9],
              gradient=False)


def test_thousands_of_sequences():
    """Short sequences, some empty, some padded, several to a block."""
    rng = np.random.default_rng(3)
    T, S, E = 20000, 4096, 40
    l, ids = problem(3, T, E, 2, torch.bfloat16)
    cuts = np.sort(rng.integers(0, T + 1, S + 1)).tolist()
    lens = rng.integers(0, 9, S).tolist()
    say("balance of thousands of sequences")
    check(l, ids, "softmax", cuts, gradient=False)
    check(l, ids, "sigmoid", cuts, lens, gradient=False)
    r = mxq.moe_balance_loss(l, ids, seq_offsets=i32_to_dev(cuts))
    g = rng.standard_normal(S).astype(np.float32)
    out = mxq.moe_balance_loss_backward(f32_to_dev(g), l, r["counts"],
                                        seq_offsets=i32_to_dev(cuts))
    want, err = mx.balance_backward(g, None, l.double().cpu().numpy(),
                                    host(r["counts"]), "softmax", cuts, None,
                                    S)
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= err + HALF[out.dtype] * (np.abs(want) + err)).all()
