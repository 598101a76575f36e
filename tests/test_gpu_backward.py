"""moe_scatter_rows_backward and moe_combine_backward against the 64-bit
reference.

Tolerances: the sort's gradient adds K values in fp32, each addition off by
at most 2^-24 of the running sum's size, which is at most the sum of the
absolute values; then one rounding to the output's type.  grad_y is one
product rounded to fp32 and to bf16.  grad_weights adds H products by fused
multiply-adds: each lane's eight partial sums take H / 512 of them in order,
joined by nine additions, each off by at most 2^-24 of the sum of absolute
products."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import operator_refs as ref
import synthetic_inputs as si
from gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def routing(T, K, E, n_local, seed):
    """Compact layout of a routing whose last experts lie elsewhere."""
    ids = si.uniform_topk(np.random.default_rng(seed), T, E, K)
    lay = mxq.moe_layout(torch.from_numpy(ids).to(DEV), 0, n_local)
    return lay


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g)


SIZES = [(1, 1, 1, 1, 8), (1, 8, 256, 256, 7168), (3, 2, 8, 3, 1032),
         (130, 5, 9, 9, 520), (193, 8, 64, 8, 1024), (64, 64, 64, 64, 16),
         (300, 9, 20, 20, 2056), (20, 3, 4, 4, 32768)]


@pytest.mark.parametrize("tin,tout", [("bf16", "bf16"), ("bf16", "f32"),
                                      ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,K,E,local,H", SIZES)
def test_scatter_rows_backward(T, K, E, local, H, tin, tout):
    lay = routing(T, K, E, local, T + H)
    rows = randn(T, lay["num_rows"], H).to(TYPES[tin])
    say("scatter_rows_backward", T, K, E, local, H, tin, tout)
    out = mxq.moe_scatter_rows_backward(rows.to(DEV), lay["src2dst"],
                                        out_dtype=TYPES[tout])
    assert out.dtype == TYPES[tout]
    s = host(lay["src2dst"])
    want = ref.scatter_rows_backward(rows.double().numpy(), s)
    size = ref.scatter_rows_backward(rows.double().abs().numpy(), s)
    err = np.abs(out.cpu().double().numpy() - want)
    assert (err <= HALF[tout] * np.abs(want) * 1.01 +
            K * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("tg", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,local,H", SIZES)
def test_combine_backward(T, K, E, local, H, tg):
    lay = routing(T, K, E, local, T + H)
    R = lay["num_rows"]
    g = randn(T, T, H).to(TYPES[tg])
    y = randn(T + 1, R, H).to(torch.bfloat16)
    w = randn(T + 2, T, K)
    gy = torch.full((R, H), 7.0, dtype=torch.bfloat16, device=DEV)
    say("combine_backward", T, K, E, local, H, tg)
    got_y, got_w = mxq.moe_combine_backward(
        g.to(DEV), y.to(DEV), lay["src2dst"], w.to(DEV), grad_y=gy)
    s = host(lay["src2dst"])
    want_y, want_w = ref.combine_backward(g.double().numpy(),
                                          y.double().numpy(), s, w.numpy(),
                                          np.full((R, H), 7.0))
    _, size = ref.combine_backward(g.double().abs().numpy(),
                                   y.double().abs().numpy(), s, w.numpy(),
                                   np.zeros((R, H)))
    np.testing.assert_allclose(got_y.cpu().double().numpy(), want_y,
                               rtol=2.0 ** -8 + 2.0 ** -23, atol=1e-40)
    err = np.abs(host(got_w).astype(np.float64) - want_w)
    assert (err <= (H / 512 + 10) * 2.0 ** -24 * size).all()
    none = s < 0
    assert (host(got_w)[none] == 0).all()


def test_gradients_are_the_transposed_maps():
    """<combine(y), g> has the slopes that the gradient says, by
    differences in fp32 outputs; and the sort's gradient is the transpose of
    moe_scatter_rows."""
    T, K, E, H = 12, 3, 5, 64
    lay = routing(T, K, E, E, 1)
    R = lay["num_rows"]
    y = randn(1, R, H).to(torch.bfloat16).to(DEV)
    w = torch.rand((T, K), device=DEV)
    g = randn(2, T, H).to(DEV)
    gy, gw = mxq.moe_combine_backward(g, y, lay["src2dst"], w)
    out = mxq.moe_combine(y, lay["src2dst"], w, out_dtype=torch.float32)
    for t, j in ((0, 0), (5, 2), (11, 1)):
        w2 = w.clone()
        w2[t, j] += 1.0  # the combine is linear in its weights
        out2 = mxq.moe_combine(y, lay["src2dst"], w2,
                               out_dtype=torch.float32)
        slope = ((out2.double() - out.double()) * g.double()).sum()
        # both outputs are off by K steps of 2^-24 of their size, at most
        # K * 2 * 4.5 for weights below 2 and normal y; |g| < 4.5, H of them
        size = K * 2 * 4.5
        assert abs(slope.item() - gw[t, j].item()) < \
            H * 4.5 * 2 * K * 2.0 ** -24 * size
    x = randn(3, T, H).to(DEV)
    rows, _ = mxq.moe_scatter_rows(x.view(torch.uint8), lay["src2dst"], R)
    rows = rows.view(torch.float32)
    d = lay["src2dst"].long().reshape(-1)
    r = randn(4, R, H).to(DEV)
    gx = mxq.moe_scatter_rows_backward(r, lay["src2dst"])
    a = (rows[d].double() * r[d].double()).sum()
    b = (x.double() * gx.double()).sum()
    # every gx is off by at most K steps of 2^-24 of its absolute terms
    size = torch.from_numpy(ref.scatter_rows_backward(
        r.cpu().double().abs().numpy(), host(lay["src2dst"])))
    bound = K * 2.0 ** -24 * (x.cpu().double().abs() * size).sum()
    assert abs((a - b).item()) <= bound.item()


def test_padding_never_read_and_bad_indices_skipped():
    T, K, H, R = 6, 4, 256, 40
    s = torch.tensor([[0, 5, -1, 39], [40, 1 << 30, -7, 2], [-1] * 4,
                      [10, 11, 12, 13], [20, -1, 21, -1], [30, 31, 32, 33]],
                     dtype=torch.int32, device=DEV)
    live = [d for d in s.flatten().tolist() if 0 <= d < R]
    rows = torch.full((R, H), float("nan"))
    rows[live] = randn(1, len(live), H)
    y = rows.to(torch.bfloat16)
    g, w = randn(2, T, H), randn(3, T, K)
    out = mxq.moe_scatter_rows_backward(rows.to(DEV), s)
    want = ref.scatter_rows_backward(rows.double().numpy(), host(s))
    np.testing.assert_allclose(out.cpu().double().numpy(), want, atol=4e-6)
    assert (out[2] == 0).all()
    gy0 = torch.full((R, H), 9.0, dtype=torch.bfloat16, device=DEV)
    gy, gw = mxq.moe_combine_backward(g.to(DEV), y.to(DEV), s, w.to(DEV),
                                      grad_y=gy0)
    wy, ww = ref.combine_backward(g.numpy(), y.double().numpy(), host(s),
                                  w.numpy(), np.full((R, H), 9.0))
    np.testing.assert_allclose(gy.cpu().double().numpy(), wy,
                               rtol=2.0 ** -8 + 2.0 ** -23)
    np.testing.assert_allclose(host(gw), ww, atol=256 * 16 * 2.0 ** -24)


def test_strides():
    T, K, E, H = 50, 4, 6, 264
    lay = routing(T, K, E, E, 7)
    R = lay["num_rows"]
    s = lay["src2dst"]
    big = randn(1, R, H + 24).to(torch.bfloat16).to(DEV)
    rows = big[:, 8:8 + H]
    a = mxq.moe_scatter_rows_backward(rows, s)
    b = mxq.moe_scatter_rows_backward(rows.contiguous(), s)
    assert torch.equal(a, b)
    out = torch.full((T + 2, H + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    mxq.moe_scatter_rows_backward(rows, s, out=out[:, :H])
    assert torch.equal(out[:T, :H], b)
    assert (out[T:] == 3).all() and (out[:, H:] == 3).all()
    g = randn(2, T, H + 8).to(DEV)[:, :H]
    w = randn(3, T, K).to(DEV)
    gy = torch.full((R, H + 16), 3.0, dtype=torch.bfloat16, device=DEV)
    _, gw = mxq.moe_combine_backward(g, rows, s, w, grad_y=gy[:, :H])
    ry, rw = mxq.moe_combine_backward(g.contiguous(), rows.contiguous(), s, w)
    d = s.long().flatten()
    assert torch.equal(gy[:, :H][d], ry[d]) and torch.equal(gw, rw)
    assert (gy[:, H:] == 3).all()


def test_empty():
    s = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    rows = torch.zeros((16, 64), device=DEV)
    assert mxq.moe_scatter_rows_backward(rows, s).shape == (0, 64)
    y = rows.bfloat16()
    w = torch.empty((0, 4), device=DEV)
    gy, gw = mxq.moe_combine_backward(rows[:0], y, s, w)
    assert gw.shape == (0, 4)
    # no rows at all on this rank
    s = torch.full((5, 4), -1, dtype=torch.int32, device=DEV)
    none = torch.empty((0, 64), device=DEV)
    assert (mxq.moe_scatter_rows_backward(none, s) == 0).all()
    gy, gw = mxq.moe_combine_backward(
        torch.ones((5, 64), device=DEV), none.bfloat16(), s,
        torch.ones((5, 4), device=DEV))
    assert gy.shape == (0, 64) and (gw == 0).all()


def test_refusals():
    s = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    y = torch.zeros((8, 64), dtype=torch.bfloat16, device=DEV)
    g = torch.zeros((4, 64), device=DEV)
    w = torch.zeros((4, 2), device=DEV)
    with pytest.raises(TypeError):
        mxq.moe_scatter_rows_backward(y.half(), s)
    with pytest.raises(mxq.MxqError):
        mxq.moe_scatter_rows_backward(y[:, 1:57], s)   # not on 16 bytes
    with pytest.raises(mxq.MxqError):
        mxq.moe_scatter_rows_backward(y[:, :60].contiguous(), s)
    with pytest.raises(ValueError):
        mxq.moe_scatter_rows_backward(y, s, out=y[:3])
    with pytest.raises(ValueError):
        mxq.moe_scatter_rows_backward(y, s.long())
    with pytest.raises(TypeError):
        mxq.moe_combine_backward(g, y.float(), s, w)
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y[:, :56], s, w)
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g[:3], y, s, w)
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y, s, w.double())
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y, s, w, grad_y=y[:7])
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(g, y, s, w.cpu())


def test_rows_beyond_32_bit_offsets():
    """Destinations past 2^32 bytes of the rows' start."""
    T, K, H, rows = 40, 3, 8192, 300000
    src = torch.arange(T * K, dtype=torch.int32).view(T, K)
    far = (rows - T * K + src).to(DEV)
    near = src.to(DEV)
    y = randn(1, T * K, H).bfloat16().to(DEV)
    big = torch.empty((rows, H), dtype=torch.bfloat16, device=DEV)
    big[rows - T * K:] = y
    g = randn(2, T, H).bfloat16().to(DEV)
    w = randn(3, T, K).to(DEV)
    say("rows beyond 32-bit offsets")
    gy, gw = mxq.moe_combine_backward(g, y, near, w)
    far_gy, far_gw = mxq.moe_combine_backward(g, big, far, w)
    assert torch.equal(far_gw, gw)
    assert torch.equal(far_gy[rows - T * K:], gy)
    assert torch.equal(mxq.moe_scatter_rows_backward(big, far),
                       mxq.moe_scatter_rows_backward(y, near))


def test_sort_gradient_of_very_wide_rows():
    """More channels than 65535 blocks of the usual size."""
    H = 70000 * 1024 + 8
    rows = (torch.arange(2 * H, device=DEV) % 251 - 125).bfloat16().view(2, H)
    s = torch.tensor([[0, 1, -1]], dtype=torch.int32, device=DEV)
    say("very wide rows")
    out = mxq.moe_scatter_rows_backward(rows, s)
    assert torch.equal(out[0], rows[0] + rows[1])  # whole numbers below 256


@pytest.mark.parametrize("H,tg", [(8, "f32"), (520, "bf16"), (1528, "f32"),
                                  (7168, "bf16"), (16384, "f32")])
def test_combine_backward_by_rows_here(H, tg):
    """Tokens with none to all of nine assignments here: the shares of a row
    that wavefronts take.  The bound is test_combine_backward's: with p
    vectors of 512 channels a row's sum has at most p fused steps and joins
    of shares, and nine joins within a wavefront."""
    T, K = 80, 9
    rng = np.random.default_rng(H)
    s = np.full((T, K), -1, np.int32)
    rows = rng.permutation(T * K)
    at = 0
    for t in range(T):
        here = rng.permutation(K)[:t % (K + 1)]
        s[t, here] = rows[at:at + len(here)]
        at += len(here)
    g = randn(1, T, H).to(TYPES[tg])
    y = randn(2, T * K, H).bfloat16()
    w = randn(3, T, K)
    say("combine_backward by rows here", H, tg)
    src = torch.from_numpy(s).to(DEV)
    fill = torch.full((T * K, H), 7.0, dtype=torch.bfloat16, device=DEV)
    got_w = torch.full((T, K), 7.0, device=DEV)
    got_y, _ = mxq.moe_combine_backward(g.to(DEV), y.to(DEV), src, w.to(DEV),
                                        grad_y=fill, grad_weights=got_w)
    want_y, want_w = ref.combine_backward(
        g.double().numpy(), y.double().numpy(), s, w.numpy(),
        np.full((T * K, H), 7.0))
    _, size = ref.combine_backward(
        g.double().abs().numpy(), y.double().abs().numpy(), s, w.numpy(),
        np.zeros((T * K, H)))
    np.testing.assert_allclose(got_y.cpu().double().numpy(), want_y,
                               rtol=2.0 ** -8 + 2.0 ** -23, atol=1e-40)
    err = np.abs(host(got_w).astype(np.float64) - want_w)
    assert (err <= (H / 512 + 10) * 2.0 ** -24 * size).all()
    assert (host(got_w)[s < 0] == 0).all()
