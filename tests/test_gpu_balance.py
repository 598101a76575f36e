"""moe_balance_loss and its gradient against the 64-bit reference.  The
tolerances are the reference's bounds of what fp32 exponentials and sums make
of the shares, plus half a step of the output's type."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import mx_refs as mx
from gpu_util import DEV, assert_equal, f32_to_dev, host, i32_to_dev, say

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def check(logits, ids, scoring, offsets=None, lens=None, z=True, add=None,
          seed=0):
    """Forward and backward of one call; returns the outputs."""
    S = 1 if offsets is None else len(offsets) - 1
    L = logits.double().cpu().numpy()
    T, E = L.shape
    kw = dict(scoring=scoring,
              seq_offsets=None if offsets is None else i32_to_dev(offsets),
              seq_lens=None if lens is None else i32_to_dev(lens))
    r = mxq.moe_balance_loss(logits, ids, z_loss=z, **kw)
    loss, zl, counts, probs, perr, zerr = mx.balance(
        L, host(ids), scoring, offsets, lens, S)
    assert_equal(host(r["counts"]), counts.astype(np.int32), "counts")
    got = host(r["probs"])
    assert (np.abs(got - probs) <= perr + 2.0 ** -24 * probs).all()
    total = np.maximum(counts.sum(1), 1)
    lerr = E * (counts * perr).sum(1) / total
    got = host(r["loss"])
    assert (np.abs(got - loss) <= lerr + 2.0 ** -24 * loss).all()
    assert ("z_loss" in r) == z
    if z:
        assert (np.abs(host(r["z_loss"]) - zl) <= zerr).all()
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(S).astype(np.float32) * T
    gz = rng.standard_normal(S).astype(np.float32) * T if z else None
    out = mxq.moe_balance_loss_backward(
        f32_to_dev(g), logits, r["counts"], add=add,
        grad_z=None if gz is None else f32_to_dev(gz), **kw)
    want, err = mx.balance_backward(
        g, gz, L, counts, scoring, offsets, lens, S,
        None if add is None else add.double().cpu().numpy())
    assert out.dtype == logits.dtype
    off = np.abs(out.double().cpu().numpy() - want)
    lim = err + HALF[out.dtype] * (np.abs(want) + err)
    assert (off <= lim).all(), (off / lim).max()
    return r, out


def problem(seed, T, E, K, dtype=torch.float32, spread=2.0, dead=0):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn((T, E), generator=g) * spread).to(dtype)
    if dead:
        l[:, torch.randperm(E, generator=g)[:dead]] = float("-inf")
    ids = l.float().topk(K, 1).indices.int()
    return l.to(DEV), ids.to(DEV)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [
    (1, 1, 1), (1, 4, 2), (3, 5, 3), (17, 16, 4), (64, 17, 1), (65, 33, 8),
    (130, 64, 2), (63, 65, 5), (64, 129, 6), (65, 256, 8), (70, 257, 4),
    (40, 512, 3), (9, 513, 7), (33, 1000, 10), (12, 1024, 64)])
def test_sizes(T, E, K, dtype, scoring):
    say("balance", T, E, K, dtype, scoring)
    l, ids = problem(T + E, T, E, K, dtype)
    check(l, ids, scoring)
    check(l, ids, scoring, z=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(600, 8), (1025, 12), (900, 130),
                                 (520, 600)])
def test_two_launches(T, E, scoring):
    """More tokens than one launch takes, alone and in sequences that begin
    and end inside a block's tokens."""
    assert mxq.moe_balance_loss_workspace_bytes(max(T, 2000), E, 1) > 0
    l, ids = problem(T, T, E, 3, torch.bfloat16)
    say("balance two launches", T, E, scoring)
    check(l, ids, scoring)
    cuts = [0, 1, 1, 40, 41, 300, T - 7, T]
    check(l, ids, scoring, cuts)
    check(l, ids, scoring, cuts, [1, 0, 20, 9, 100, 0, 7])


def test_many_sequences():
    """More sequences than a wavefront, or a block, has lanes."""
    for S, T in ((70, 200), (600, 1500), (1300, 1300)):
        l, ids = problem(S, T, 10, 2)
        rng = np.random.default_rng(S)
        cuts = np.sort(rng.integers(0, T + 1, S - 1)).tolist()
        say("balance sequences", S, T)
        r, _ = check(l, ids, "softmax", [0] + cuts + [T])
        assert int(r["counts"].sum()) == 2 * T


def test_padding_and_empty():
    l, ids = problem(5, 300, 20, 2)
    add = (torch.randn((300, 20), device=DEV) * 3)
    # tokens before the first sequence, behind the last, and of none between
    _, g = check(l, ids, "softmax", [10, 40, 40, 250], [25, 3, 200], add=add)
    for a, b in ((0, 10), (35, 40), (240, 300)):
        assert torch.equal(g[a:b], add[a:b])
    _, g = check(l, ids, "sigmoid", [10, 40, 40, 250], [25, 3, 200])
    assert (g[35:40] == 0).all()
    # one sequence with a length, without offsets
    _, g = check(l, ids, "softmax", None, [123], add=add)
    assert torch.equal(g[123:], add[123:])
    # no token at all
    r, g = check(l[:0], ids[:0], "softmax")
    assert (host(r["loss"]) == 0).all() and g.shape == (0, 20)
    r, _ = check(l, ids, "softmax", [0, 0, 300], [0, 0])
    assert not r["counts"].any() and not r["probs"].any()


def test_offsets_out_of_range():
    """Offsets and lengths that no batch makes: cut to the tokens."""
    l, ids = problem(6, 500, 40, 3)
    for off, lens in (([-5, 100, 1 << 30], None),
                      ([0, 200, 400], [1 << 30, -3]),
                      ([600, 700, 800], None)):
        check(l, ids, "softmax", off, lens)
    # descending ones: unspecified, but nothing outside is touched
    r = mxq.moe_balance_loss(l, ids, seq_offsets=i32_to_dev([400, 10, 300]))
    mxq.moe_balance_loss_backward(torch.ones(2, device=DEV), l, r["counts"],
                                  seq_offsets=i32_to_dev([400, 10, 300]))
    torch.cuda.synchronize()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_special_logits(scoring):
    """Dead experts and rows, NaN, infinities, far logits, missing ids."""
    l, ids = problem(7, 90, 24, 4, dead=5)
    l[3] = float("-inf")
    l[5, 7] = float("nan")
    l[8] = float("nan")
    l[9] *= 20
    l[10] -= 200          # sigmoids below fp32
    l[11] = 0.0
    l[12, 0] = 60.0       # one share is nearly all
    ids[3] = -1
    ids[6, 1] = 24
    ids[7] = 2            # the same expert four times
    r, g = check(l, ids, scoring)
    dead = ~(l > float("-inf"))
    assert (g[dead] == 0).all() and torch.isfinite(g).all()
    # +inf counts as the largest finite value; its square is beyond fp32
    l[13, 4] = float("inf")
    r, g = check(l, ids, scoring, z=False)
    assert torch.isfinite(r["loss"]).all() and torch.isfinite(g).all()


def test_saturated_shares_keep_their_bits():
    """A share of nearly one, whose difference to one fp32 does not hold: the
    gradient is of what the others have."""
    l = torch.zeros((4, 16), device=DEV)
    l[:, 3] = 30.0
    ids = torch.arange(16, device=DEV, dtype=torch.int32).reshape(4, 4)
    ids[0] = 3
    r, g = check(l, ids, "softmax", z=False)
    assert (g[:, 3] != 0).all()


def test_counts_of_other_ranks():
    """Counts summed over ranks, up to where 32 bits end."""
    l, _ = problem(8, 50, 12, 2)
    L = l.double().cpu().numpy()
    g = np.array([50.0], np.float32)
    for counts in (np.arange(12) * 1000, np.zeros(12, int),
                   np.array([2 ** 31 - 1, 0] + [5] * 10)):
        counts = counts.reshape(1, 12).astype(np.int64)
        out = mxq.moe_balance_loss_backward(f32_to_dev(g), l,
                                            i32_to_dev(counts))
        want, err = mx.balance_backward(g, None, L, counts, "softmax")
        off = np.abs(host(out) - want)
        assert (off <= err + 2.0 ** -24 * np.abs(want)).all()


def test_gradients_apart_and_together():
    l, ids = problem(9, 200, 30, 2)
    r = mxq.moe_balance_loss(l, ids, z_loss=True)
    one = torch.full((1,), 300.0, device=DEV)
    a = mxq.moe_balance_loss_backward(one, l, r["counts"])
    b = mxq.moe_balance_loss_backward(None, l, None, grad_z=one)
    c = mxq.moe_balance_loss_backward(one, l, r["counts"], grad_z=one)
    want, _ = mx.balance_backward(None, host(one), l.double().cpu().numpy(),
                                  host(r["counts"]), "softmax")
    assert np.abs(host(b) - want).max() <= 1e-5 * np.abs(want).max()
    # three roundings of fp32 more or less
    assert ((a + b - c).abs() <= 3 * 2.0 ** -24 *
            (a.abs() + b.abs())).all()
    # in place over the router's gradient
    add = torch.randn((200, 30), device=DEV)
    want = mxq.moe_balance_loss_backward(one, l, r["counts"], add=add)
    out = mxq.moe_balance_loss_backward(one, l, r["counts"], add=add,
                                        grad_logits=add)
    assert out is add and torch.equal(add, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides(dtype):
    for E in (20, 21, 160):
        l, ids = problem(10, 100, E, 2, dtype)
        add = torch.randn((100, E), device=DEV).to(dtype)
        r = mxq.moe_balance_loss(l, ids, z_loss=True)
        one = torch.ones(1, device=DEV) * 100
        want = mxq.moe_balance_loss_backward(one, l, r["counts"], grad_z=one,
                                             add=add)

        def wide(t, left, right):
            big = torch.full((t.shape[0], left + t.shape[1] + right), 7.0,
                             dtype=t.dtype, device=DEV)
            v = big[:, left:left + t.shape[1]]
            v.copy_(t)
            return v, big

        for left in (8, 3):
            lw, _ = wide(l, left, 5)
            aw, _ = wide(add, left, 2)
            out, big = wide(torch.zeros_like(l), left, 8)
            r2 = mxq.moe_balance_loss(lw, ids, z_loss=True)
            for k in r:
                assert torch.equal(r[k], r2[k]), k
            mxq.moe_balance_loss_backward(one, lw, r2["counts"], grad_z=one,
                                          add=aw, grad_logits=out)
            assert torch.equal(out, want)
            assert (big[:, :left] == 7).all()
            assert (big[:, left + E:] == 7).all()


def test_many_tokens():
    """Blocks with several rounds each; fixed order: equal calls, equal
    bytes."""
    T, E, K = 40000, 96, 4
    l, ids = problem(11, T, E, K, torch.bfloat16)
    off = [0, 100, 17000, 17001, 39990]
    r, g = check(l, ids, "softmax", off)
    for _ in range(3):
        r2 = mxq.moe_balance_loss(l, ids, seq_offsets=i32_to_dev(off),
                                  z_loss=True)
        for k in r:
            assert torch.equal(r[k], r2[k]), k


def test_graph_and_streams():
    """Captured with a workspace of its own, replayed with new inputs; and
    two streams at once."""
    T, E, K = 3000, 64, 4
    l, ids = problem(12, T, E, K)
    off = i32_to_dev([0, 1000, 2500])
    ws = torch.empty(mxq.moe_balance_loss_workspace_bytes(T, E, 2),
                     dtype=torch.uint8, device=DEV)
    grad = torch.ones(2, device=DEV) * 1000

    def step(w):
        r = mxq.moe_balance_loss(l, ids, "sigmoid", off, z_loss=True,
                                 workspace=w)
        g = mxq.moe_balance_loss_backward(grad, l, r["counts"], "sigmoid",
                                          off, grad_z=grad)
        return r, g

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws)
    torch.cuda.current_stream().wait_stream(side)
    graph, twin = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, g = step(ws)
    with torch.cuda.graph(twin):   # a second graph over the same workspace
        r2, g2 = step(ws)
    for i in range(3):
        say("balance replay", i)
        a, b = problem(100 + i, T, E, K)
        l.copy_(a)
        ids.copy_(b)
        graph.replay()
        twin.replay()
        torch.cuda.synchronize()
        want, wg = step(None)
        for k in want:
            assert torch.equal(r[k], want[k]) and torch.equal(r2[k], want[k])
        assert torch.equal(g, wg) and torch.equal(g2, wg)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step(None))
    torch.cuda.synchronize()
    for o, og in outs:
        assert torch.equal(og, wg) and torch.equal(o["loss"], want["loss"])


def test_with_the_router():
    """A router's training step: the weights' gradient and the loss's in one
    buffer, against the sum of both."""
    T, E, K = 500, 48, 4
    l, _ = problem(13, T, E, K)
    ids, w = mxq.moe_route(l, K, scoring="sigmoid")
    gw = torch.randn((T, K), device=DEV)
    r = mxq.moe_balance_loss(l, ids, "sigmoid")
    lay = mxq.moe_layout(ids, 0, E)
    assert torch.equal(r["counts"][0], lay["counts"])
    route = mxq.moe_route_backward(gw, l, ids, scoring="sigmoid")
    one = torch.full((1,), 0.01 * T, device=DEV)
    want, err = mx.balance_backward(
        host(one), None, l.double().cpu().numpy(), host(r["counts"]),
        "sigmoid", add=host(route).astype(np.float64))
    got = host(mxq.moe_balance_loss_backward(
        one, l, r["counts"], "sigmoid", add=route, grad_logits=route))
    assert (np.abs(got - want) <= err + 2.0 ** -24 * np.abs(want)).all()


def test_refusals():
    l, ids = problem(14, 2000, 20, 2)
    r = mxq.moe_balance_loss(l, ids)
    one = torch.ones(1, device=DEV)
    off = i32_to_dev([0, 5, 9])
    for f in (lambda: mxq.moe_balance_loss(l, ids.long()),
              lambda: mxq.moe_balance_loss(l, ids[:, 0]),
              lambda: mxq.moe_balance_loss(l, ids[:50]),
              lambda: mxq.moe_balance_loss(l, ids, seq_offsets=off.long()),
              lambda: mxq.moe_balance_loss(l, ids, seq_offsets=off[:1]),
              lambda: mxq.moe_balance_loss(l, ids, seq_offsets=off,
                                           seq_lens=i32_to_dev([1])),
              lambda: mxq.moe_balance_loss(l, ids, out=dict(loss=one[:0])),
              lambda: mxq.moe_balance_loss(l, ids, workspace=one),
              lambda: mxq.moe_balance_loss(l.cpu(), ids),
              lambda: mxq.moe_balance_loss(l, ids.cpu()),
              lambda: mxq.moe_balance_loss_backward(None, l, r["counts"]),
              lambda: mxq.moe_balance_loss_backward(one, l, r["counts"][0]),
              lambda: mxq.moe_balance_loss_backward(one, l, r["counts"],
                                                    seq_offsets=off),
              lambda: mxq.moe_balance_loss_backward(one, l, r["counts"],
                                                    add=l[:9])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        mxq.moe_balance_loss(l.half(), ids)
    with pytest.raises(TypeError):
        mxq.moe_balance_loss_backward(one, l, r["counts"], add=l.bfloat16())
    with pytest.raises(KeyError):
        mxq.moe_balance_loss(l, ids, scoring="relu")
    with pytest.raises(mxq.MxqError):   # counts are needed
        mxq.moe_balance_loss_backward(one, l, None)
    with pytest.raises(mxq.MxqError):   # a short workspace
        mxq.moe_balance_loss(l, ids, workspace=torch.empty(
            16, dtype=torch.uint8, device=DEV))
