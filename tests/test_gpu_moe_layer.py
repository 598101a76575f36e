"""The router, the layout, the experts' products, the combine and the
gradients in a row, as a layer runs them: a forward pass against the 64-bit
definition, a training step's gradients, both captured in one graph and
replayed with new inputs, and two streams at once."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import operator_refs as ref
from gpu_util import DEV, assert_equal, host, say

pytestmark = pytest.mark.gpu

GROUP = {"ue8m0_g128": 128, "e8m0_g32": 32}


class Layer:
    """Weights of one layer: fp8 with block scales, as
    requant_weight_block_ue8m0 makes them from scaled fp8 weights."""

    def __init__(self, seed, E, H, I):
        g = torch.Generator().manual_seed(seed)
        self.E, self.H, self.I = E, H, I

        def weights(n, k):
            q = (torch.randn((E, n, k), generator=g) * 64).clamp(-448, 448)
            q = q.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
            s = torch.full((E, -(-n // 128), -(-k // 128)),
                           1.0 / (64 * k ** 0.5), device=DEV)
            return mxq.requant_weight_block_ue8m0(q, s)

        self.w1, self.s1 = weights(2 * I, H)
        self.w2, self.s2 = weights(H, I)


def forward(L, x, logits, K, kind, fmt, m):
    """One pass, every call on the current stream."""
    T = x.shape[0]
    ids, w = mxq.moe_route(logits, K, scoring="sigmoid", weight_scale=1.5)
    lay = mxq.moe_layout(ids, 0, L.E, kind, capacity=128 * -(-T // 128))
    q, s = mxq.moe_scatter_quant_ex(x, lay["src2dst"], lay["num_rows"],
                                    fmt=fmt)
    n = lay["masked_m"] if kind == "masked" else lay["counts"]
    hq, hs = mxq.moe_expert_matmul_quant(q, s, L.w1, L.s1,
                                         lay["expert_offsets"], n, fmt=fmt,
                                         out_fmt=fmt, expected_m=m)
    y = mxq.moe_expert_matmul(hq, hs, L.w2, L.s2, lay["expert_offsets"], n,
                              fmt=fmt, expected_m=m)
    out = mxq.moe_combine(y, lay["src2dst"], w, out_dtype=torch.float32)
    return dict(ids=ids, w=w, lay=lay, q=q, s=s, hq=hq, hs=hs, y=y, out=out,
                n=n)


def check_forward(L, x, logits, K, fmt, r):
    """Each step against the definition, from the bytes the step before it
    wrote."""
    G = GROUP[fmt]
    rid, rw = ref.route(logits.double().cpu().numpy(), K, scoring="sigmoid",
                        scale=1.5)
    assert_equal(host(r["ids"]), rid, "ids")
    np.testing.assert_allclose(host(r["w"]), rw, rtol=2.0 ** -24 * 1.001)
    off, n = host(r["lay"]["expert_offsets"]), host(r["n"])
    rows = r["lay"]["num_rows"]
    live = np.zeros(rows, bool)
    for e in range(L.E):
        live[off[e]:off[e] + n[e]] = True
    assert live.sum() == (rid >= 0).sum()
    q, s = host(r["q"]).copy(), host(r["s"]).copy()
    h, herr = ref.expert_matmul(q, s, G, host(L.w1), host(L.s1), off, n, None,
                                "silu_mul", None, L.I)
    hq, hs = host(r["hq"]), host(r["hs"])
    ref.check_quantized(h, herr, hq, hs, G, live)
    y, yerr = ref.expert_matmul(hq, hs, G, host(L.w2), host(L.s2), off, n,
                                None, "none", None, L.H)
    got = r["y"].double().cpu().numpy()
    lim = 2.0 ** -8 * (np.abs(y) + yerr) + yerr
    assert (np.abs(got - y)[live] <= lim[live]).all()
    src, w = host(r["lay"]["src2dst"]), host(r["w"]).astype(np.float64)
    out = host(r["out"])
    for t in range(x.shape[0]):
        d = src[t]
        terms = [(w[t, j], got[d[j]]) for j in range(K) if d[j] >= 0]
        want = sum(a * b for a, b in terms)
        size = sum(abs(a) * np.abs(b) for a, b in terms)
        assert (np.abs(out[t] - want) <= K * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("kind", ["compact", "masked"])
@pytest.mark.parametrize("fmt,H,I", [("ue8m0_g128", 512, 256),
                                     ("e8m0_g32", 416, 160)])
@pytest.mark.parametrize("T,m", [(1, 1), (40, None), (300, 1 << 20)])
def test_forward(T, m, fmt, H, I, kind):
    say("layer", T, m, fmt, H, I, kind)
    L = Layer(1, 8, H, I)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).bfloat16().to(DEV)
    logits = torch.randn((T, 8), generator=g).to(DEV)
    logits[:, 3] = float("-inf")     # an expert out of service
    r = forward(L, x, logits, 3, kind, fmt, m)
    check_forward(L, x, logits, 3, fmt, r)


def test_forward_with_fewer_experts_than_choices():
    """Ids of -1 pass through the layout, the products and the combine."""
    L = Layer(2, 8, 256, 128)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((50, 256), generator=g).bfloat16().to(DEV)
    logits = torch.randn((50, 8), generator=g).to(DEV)
    logits[:25, 2:] = float("-inf")
    logits[7] = float("-inf")
    r = forward(L, x, logits, 4, "compact", "ue8m0_g128", None)
    check_forward(L, x, logits, 4, "ue8m0_g128", r)
    assert (host(r["ids"])[7] == -1).all()
    assert (host(r["out"])[7] == 0).all()


def training_step(x, y, lay, logits, ids, w, g, out):
    """Gradients of sum(g * combine(y, route(logits))) and of the sort."""
    gy, gw = mxq.moe_combine_backward(g, y, lay["src2dst"], w,
                                      grad_y=out["gy"],
                                      grad_weights=out["gw"])
    gl = mxq.moe_route_backward(gw, logits, ids, scoring="sigmoid",
                                weight_scale=1.5, grad_logits=out["gl"])
    gx = mxq.moe_scatter_rows_backward(gy, lay["src2dst"], out=out["gx"])
    return gy, gw, gl, gx


def test_training_step_gradients():
    T, E, K, H = 60, 12, 4, 264
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((T, E), generator=g).to(DEV)
    ids, w = mxq.moe_route(logits, K, scoring="sigmoid", weight_scale=1.5)
    lay = mxq.moe_layout(ids, 0, E)
    R = lay["num_rows"]
    y = torch.randn((R, H), generator=g).bfloat16().to(DEV)
    go = torch.randn((T, H), generator=g).to(DEV)
    out = dict(gy=torch.zeros_like(y), gw=torch.zeros_like(w),
               gl=torch.zeros_like(logits),
               gx=torch.zeros((T, H), dtype=torch.bfloat16, device=DEV))
    gy, gw, gl, gx = training_step(None, y, lay, logits, ids, w, go, out)
    src = host(lay["src2dst"])
    wy, ww = ref.combine_backward(go.double().cpu().numpy(),
                                  y.double().cpu().numpy(), src, host(w),
                                  np.zeros((R, H)))
    np.testing.assert_allclose(gy.double().cpu().numpy(), wy,
                               rtol=2.0 ** -8 + 2.0 ** -23, atol=1e-40)
    _, size = ref.combine_backward(go.double().abs().cpu().numpy(),
                                   y.double().abs().cpu().numpy(), src,
                                   host(w), np.zeros((R, H)))
    assert (np.abs(host(gw) - ww) <= 11 * 2.0 ** -24 * size).all()
    # from here on, each step from what the step before it wrote
    wl = ref.route_backward(host(gw), logits.double().cpu().numpy(),
                            host(ids), "sigmoid", True, 1.5)
    np.testing.assert_allclose(host(gl), wl, rtol=2.0 ** -24 * 1.001,
                               atol=1.5 * np.abs(host(gw)).max() * 2.0 ** -48)
    wx = ref.scatter_rows_backward(gy.double().cpu().numpy(), src)
    sx = ref.scatter_rows_backward(gy.double().abs().cpu().numpy(), src)
    assert (np.abs(gx.double().cpu().numpy() - wx) <=
            2.0 ** -8 * np.abs(wx) * 1.01 + K * 2.0 ** -24 * sx).all()
    # the whole chain against differences of the loss in the logits
    L64 = logits.double().cpu().numpy()
    y64, g64 = y.double().cpu().numpy(), go.double().cpu().numpy()
    dots = np.einsum("tkh,th->tk", y64[src], g64)

    def loss(l):
        p = 1 / (1 + np.exp(-np.take_along_axis(l, host(ids).astype(int), 1)))
        return 1.5 * ((p / p.sum(1, keepdims=True)) * dots).sum(1)

    h = 1e-5
    for e in range(0, E, 3):
        up, dn = L64.copy(), L64.copy()
        up[:, e] += h
        dn[:, e] -= h
        slope = (loss(up) - loss(dn)) / (2 * h)
        # gw is fp32 (its error carried through factors below 1.5 / 4 each),
        # the differences are off by h^2 and 2^-52 / h of the loss
        lim = 1.5 * 11 * 2.0 ** -24 * size.sum(1) + \
            2.0 ** -24 * np.abs(wl[:, e]) + \
            (h * h + 2.0 ** -50 / h) * np.abs(dots).sum(1)
        assert (np.abs(host(gl)[:, e] - slope) <= lim).all()


@pytest.mark.parametrize("m", [1, 40, 1 << 20])
def test_graph_replays(m):
    """Forward and training step in one captured graph; new inputs are copied
    into the static buffers and eager work runs between the replays."""
    T, K, E, H, I = 48, 3, 8, 512, 256
    L = Layer(7, E, H, I)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    logits = torch.zeros((T, E), device=DEV)
    go = torch.zeros((T, H), device=DEV)
    R = mxq.moe_compact_row_bound(T * K, E)

    def step():
        r = forward(L, x, logits, K, "compact", "ue8m0_g128", m)
        out = dict(gy=gy0, gw=gw0, gl=gl0, gx=gx0)
        r["grads"] = training_step(x, r["y"], r["lay"], logits, r["ids"],
                                   r["w"], go, out)
        return r

    gy0 = torch.zeros((R, H), dtype=torch.bfloat16, device=DEV)
    gw0 = torch.zeros((T, K), device=DEV)
    gl0 = torch.zeros((T, E), device=DEV)
    gx0 = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    for i in range(4):
        say("replay", i)
        g = torch.Generator().manual_seed(100 + i)
        x.copy_(torch.randn((T, H), generator=g).bfloat16())
        logits.copy_(torch.randn((T, E), generator=g))
        go.copy_(torch.randn((T, H), generator=g))
        gy0.zero_()
        graph.replay()
        torch.cuda.synchronize()
        keys = ("ids", "w", "out")
        got = [r[k].clone() for k in keys] + [t.clone() for t in r["grads"]]
        live = r["lay"]["src2dst"].long().flatten()
        rows = [r[k][live].clone() for k in ("hq", "hs", "y")]
        gy0.zero_()
        e = step()  # eager, into the same gradient buffers
        want = [e[k] for k in keys] + list(e["grads"])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for a, k in zip(rows, ("hq", "hs", "y")):
            assert torch.equal(a, e[k][live])


def test_two_streams_at_once():
    """Calls that overlap on two streams share nothing."""
    L = Layer(11, 8, 512, 256)
    g = torch.Generator().manual_seed(1)
    jobs = []
    for T, m in ((64, 1), (200, 1 << 20)):
        x = torch.randn((T, 512), generator=g).bfloat16().to(DEV)
        logits = torch.randn((T, 8), generator=g).to(DEV)
        want = forward(L, x, logits, 3, "compact", "ue8m0_g128", m)["out"]
        jobs.append((torch.cuda.Stream(), x, logits, m, want))
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for st, x, logits, m, want in jobs:
            with torch.cuda.stream(st):
                outs.append((forward(L, x, logits, 3, "compact",
                                     "ue8m0_g128", m)["out"], want))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, b)
