"""The operators on microscaled 4-bit floats and the balance loss in a row,
as a layer runs them next to the router, the layout and the combine: a forward
pass with each step against the 64-bit definition, the balance loss's part of
the router's gradient against differences of the loss, all of it captured in
one graph and replayed with new inputs, and two streams at once; and rows
that lie far apart."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import mx_refs as mx
import operator_refs as ref
from gpu_util import DEV, assert_equal, host, i32_to_dev, say

pytestmark = pytest.mark.gpu

FMTS = ("mxfp4", "e8m0_g32")


class Layer:
    """One layer's weights, quantized from float32 master weights."""

    def __init__(self, seed, E, H, I):
        g = torch.Generator().manual_seed(seed)
        self.E, self.H, self.I = E, H, I

        def weights(n, k):
            w = torch.randn((E, n, k), generator=g) / k ** 0.5
            return mxq.mxfp4_quant_rows(w.to(DEV))

        self.w1, self.s1 = weights(2 * I, H)
        self.w2, self.s2 = weights(H, I)


def forward(L, x, logits, K, kind, fmt, mid, m, seq=None):
    """One pass with the balance loss of each sequence beside it."""
    ids, w = mxq.moe_route(logits, K, scoring="sigmoid", weight_scale=1.5)
    bal = mxq.moe_balance_loss(logits, ids, "sigmoid", seq_offsets=seq,
                               z_loss=True)
    lay = mxq.moe_layout(ids, 0, L.E, kind,
                         capacity=128 * -(-x.shape[0] // 128))
    if fmt == "mxfp4":
        q, s = mxq.moe_scatter_quant_mxfp4(x, lay["src2dst"],
                                           lay["num_rows"])
    else:
        q, s = mxq.moe_scatter_quant_ex(x, lay["src2dst"], lay["num_rows"],
                                        fmt=fmt)
    off = lay["expert_offsets"]
    n = lay["masked_m"] if kind == "masked" else lay["counts"]
    hq, hs = mxq.moe_expert_matmul_mxfp4_quant(
        q, s, L.w1, L.s1, off, n, fmt=fmt, out_fmt=mid, expected_m=m)
    y = mxq.moe_expert_matmul_mxfp4(hq, hs, L.w2, L.s2, off, n, fmt=mid,
                                    expected_m=m)
    out = mxq.moe_combine(y, lay["src2dst"], w, out_dtype=torch.float32)
    return dict(ids=ids, w=w, bal=bal, lay=lay, q=q, s=s, hq=hq, hs=hs, y=y,
                out=out, n=n)


def check_forward(L, x, logits, K, fmt, mid, r, seq=None):
    """Each step from the bytes that the step before it wrote."""
    T = x.shape[0]
    l64 = logits.double().cpu().numpy()
    ids = host(r["ids"])
    S = 1 if seq is None else len(seq) - 1
    loss, z, counts, probs, perr, zerr = mx.balance(l64, ids, "sigmoid", seq,
                                                    None, S)
    bal = {k: host(v) for k, v in r["bal"].items()}
    assert_equal(bal["counts"], counts.astype(np.int32), "counts")
    lerr = L.E * (counts * perr).sum(1) / np.maximum(counts.sum(1), 1)
    assert (np.abs(bal["loss"] - loss) <= lerr + 2.0 ** -24 * loss).all()
    assert (np.abs(bal["z_loss"] - z) <= zerr).all()
    if seq is None:
        assert_equal(bal["counts"][0], host(r["n"])[:L.E], "the layout's")
    off, n, src = (host(t) for t in (r["lay"]["expert_offsets"], r["n"],
                                     r["lay"]["src2dst"]))
    live = np.zeros(r["lay"]["num_rows"], bool)
    live[src[src >= 0]] = True
    q, s = host(r["q"]), host(r["s"])
    if fmt == "mxfp4":
        wq, ws = mx.quant(x.double().cpu().numpy())
        for j in range(K):
            ok = src[:, j] >= 0
            assert_equal(q[src[ok, j]], wq[ok], "rows")
            assert_equal(s[src[ok, j]], ws[ok], "scales")
    h, herr = mx.expert_matmul(q, s, fmt, host(L.w1), host(L.s1), off, n,
                               None, "silu_mul", None, L.I)
    hq, hs = host(r["hq"]), host(r["hs"])
    if mid == "mxfp4":
        mx.check_quantized(h, herr, hq, hs, live)
    else:
        ref.check_quantized(h, herr, hq, hs, 32, live)
    y, yerr = mx.expert_matmul(hq, hs, mid, host(L.w2), host(L.s2), off, n,
                               None, "none", None, L.H)
    got = r["y"].double().cpu().numpy()
    lim = 2.0 ** -8 * (np.abs(y) + yerr) + yerr
    assert (np.abs(got - y)[live] <= lim[live]).all()
    w, out = host(r["w"]).astype(np.float64), host(r["out"])
    for t in range(T):
        terms = [w[t, j] * got[src[t, j]] for j in range(K) if src[t, j] >= 0]
        want = sum(terms) if terms else np.zeros(L.H)
        size = sum(np.abs(v) for v in terms) if terms else np.zeros(L.H)
        assert (np.abs(out[t] - want) <= K * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("kind", ["compact", "masked"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mid", FMTS)
@pytest.mark.parametrize("T,m,H,I", [(1, 1, 512, 256), (40, None, 416, 160),
                                     (300, 1 << 20, 288, 96)])
def test_forward(T, m, H, I, mid, fmt, kind):
    say("layer", T, m, H, I, mid, fmt, kind)
    L = Layer(1, 8, H, I)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).bfloat16().to(DEV)
    logits = torch.randn((T, 8), generator=g).to(DEV)
    logits[:, 3] = float("-inf")     # an expert out of service
    r = forward(L, x, logits, 3, kind, fmt, mid, m)
    check_forward(L, x, logits, 3, fmt, mid, r)


def test_tokens_without_an_expert():
    """Ids of -1 pass through the counts, the layout and the combine."""
    L = Layer(2, 8, 256, 128)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((50, 256), generator=g).bfloat16().to(DEV)
    logits = torch.randn((50, 8), generator=g).to(DEV)
    logits[:25, 2:] = float("-inf")
    logits[7] = float("-inf")
    seq = [0, 7, 8, 8, 50]
    r = forward(L, x, logits, 4, "compact", "mxfp4", "mxfp4", None,
                i32_to_dev(seq))
    check_forward(L, x, logits, 4, "mxfp4", "mxfp4", r, seq)
    assert (host(r["ids"])[7] == -1).all()
    assert (host(r["out"])[7] == 0).all()
    assert host(r["bal"]["loss"])[1] == 0 and host(r["bal"]["loss"])[2] == 0


def gradients(logits, ids, bal, gw, gl, gz, seq, out):
    """The router's gradient and the balance loss's in one buffer."""
    mxq.moe_route_backward(gw, logits, ids, scoring="sigmoid",
                           weight_scale=1.5, grad_logits=out)
    return mxq.moe_balance_loss_backward(
        gl, logits, bal["counts"], "sigmoid", seq_offsets=seq, grad_z=gz,
        add=out, grad_logits=out)


def test_gradient_against_differences():
    """Router and balance loss together: the slope of
    sum(gw * w) + sum(gl * loss) + sum(gz * z) in the logits, the choices held
    fixed."""
    T, E, K = 60, 12, 4
    seq = [0, 25, 60]
    rng = np.random.default_rng(5)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    logits = logits.to(DEV)
    ids, _ = mxq.moe_route(logits, K, scoring="sigmoid", weight_scale=1.5)
    dseq = i32_to_dev(seq)
    bal = mxq.moe_balance_loss(logits, ids, "sigmoid", seq_offsets=dseq,
                               z_loss=True)
    gw, gl, gz = (torch.from_numpy(rng.standard_normal(n).astype(np.float32))
                  .to(DEV) for n in ((T, K), 2, 2))
    out = host(gradients(logits, ids, bal, gw, gl, gz, dseq,
                         torch.empty_like(logits)))
    l64, i = logits.double().cpu().numpy(), host(ids).astype(int)
    c = np.stack([np.bincount(i[a:b].ravel(), minlength=E)
                  for a, b in zip(seq, seq[1:])])
    gw, gl, gz = (host(t).astype(np.float64) for t in (gw, gl, gz))

    def terms(l):
        """Each token's part of the loss."""
        sig = 1 / (1 + np.exp(-l))
        p = np.take_along_axis(sig, i, 1)
        v = 1.5 * (gw * p / p.sum(1, keepdims=True)).sum(1)
        share = sig / sig.sum(1, keepdims=True)
        lse = np.log(np.exp(l).sum(1))
        for k, (a, b) in enumerate(zip(seq, seq[1:])):
            n = b - a
            v[a:b] += gl[k] * E * (share[a:b] * c[k] / c[k].sum()).sum(1) / n
            v[a:b] += gz[k] * lse[a:b] ** 2 / n
        return v

    route_err = 1.5 * np.abs(gw).max() * 2.0 ** -48
    want, err = mx.balance_backward(gl, gz, l64, c, "sigmoid", seq, None, 2)
    h = 1e-5
    for e in range(E):
        up, dn = l64.copy(), l64.copy()
        up[:, e] += h
        dn[:, e] -= h
        slope = (terms(up) - terms(dn)) / (2 * h)
        # the kernels' errors, the router's part rounded to fp32 before the
        # sum's rounding; the differences are off by h^2 of the third
        # derivative, of products of shares and values of lse^2 below 20,
        # and 2^-50 / h of the parts
        route = np.abs(slope - want[:, e])
        size = 1.5 * np.abs(gw).sum(1) + 20 * (np.abs(gl).max() +
                                               np.abs(gz).max())
        lim = err[:, e] + route_err + 2.0 ** -24 * (
            2 * route + np.abs(slope) + np.abs(want[:, e])) + \
            (20 * h * h + 2.0 ** -50 / h) * size
        assert (np.abs(out[:, e] - slope) <= lim).all(), e


@pytest.mark.parametrize("fmt,mid", [("mxfp4", "mxfp4"),
                                     ("e8m0_g32", "e8m0_g32")])
@pytest.mark.parametrize("T,m", [(48, 1), (48, 40), (700, 1 << 20)])
def test_graph_replays(T, m, fmt, mid):
    """Forward, balance loss and gradients in one captured graph, twice in two
    graphs that are replayed in turn; new inputs are copied into the static
    buffers and eager work runs between the replays."""
    K, E, H, I = 3, 8, 512, 256
    L = Layer(7, E, H, I)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    logits = torch.zeros((T, E), device=DEV)
    gw = torch.zeros((T, K), device=DEV)
    g1 = torch.zeros(1, device=DEV)

    def step():
        r = forward(L, x, logits, K, "compact", fmt, mid, m)
        r["grad"] = gradients(logits, r["ids"], r["bal"], gw, g1, g1, None,
                              torch.empty_like(logits))
        return r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = step()
        graphs.append((graph, r))

    def parts(r):
        live = r["lay"]["src2dst"].long().flatten()
        return [r[k] for k in ("ids", "w", "out", "grad")] + \
            [r["bal"][k] for k in ("loss", "z_loss", "counts", "probs")] + \
            [r[k][live] for k in ("q", "s", "hq", "hs", "y")]

    for i in range(6):
        say("replay", i)
        g = torch.Generator().manual_seed(100 + i)
        x.copy_(torch.randn((T, H), generator=g).bfloat16())
        logits.copy_(torch.randn((T, E), generator=g))
        gw.copy_(torch.randn((T, K), generator=g))
        g1.fill_(1.0 + i)
        graph, r = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in parts(r)]
        for a, b in zip(got, parts(step())):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls that overlap on two streams share nothing."""
    L = Layer(11, 8, 512, 256)
    g = torch.Generator().manual_seed(1)
    jobs = []
    for T, m, fmt in ((64, 1, "mxfp4"), (200, 1 << 20, "e8m0_g32"),
                      (6000, 18, "mxfp4")):
        x = torch.randn((T, 512), generator=g).bfloat16().to(DEV)
        logits = torch.randn((T, 8), generator=g).to(DEV)
        want = forward(L, x, logits, 3, "compact", fmt, fmt, m)
        jobs.append((torch.cuda.Stream(), x, logits, m, fmt, want))
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for st, x, logits, m, fmt, want in jobs:
            with torch.cuda.stream(st):
                outs.append((forward(L, x, logits, 3, "compact", fmt, fmt, m),
                             want))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a["out"], b["out"])
        for k in ("loss", "z_loss", "counts", "probs"):
            assert torch.equal(a["bal"][k], b["bal"][k])


def far(rows, cols, dtype):
    """Rows 65536 elements apart: offsets of the last ones pass 32 bits."""
    return torch.empty((rows, 65536), dtype=dtype, device=DEV)[:, :cols]


def test_quantization_of_rows_far_apart():
    rows, H = 66000, 64
    say("far", rows, H)
    g = torch.Generator().manual_seed(2)
    x = torch.randn((rows, H), generator=g).bfloat16().to(DEV)
    q, s = mxq.mxfp4_quant_rows(x)
    xf, qf, sf = (far(rows, n, t) for n, t in (
        (H, torch.bfloat16), (H // 2, torch.uint8), (H // 32, torch.uint8)))
    xf.copy_(x)
    mxq.mxfp4_quant_rows(xf, q=qf, scales=sf)
    assert torch.equal(qf, q) and torch.equal(sf, s)
    assert torch.equal(mxq.mxfp4_to_e4m3(qf, out=far(rows, H, torch.uint8)),
                       mxq.mxfp4_to_e4m3(q))
    assert torch.equal(mxq.upscale_mxfp4_to_bf16(qf, sf, out=xf),
                       mxq.upscale_mxfp4_to_bf16(q, s))
    # every token's rows at the ends of the buffer
    dst = torch.arange(rows, device=DEV, dtype=torch.int32)
    qf.fill_(0xA5)
    xf.copy_(x)
    src = torch.stack([dst[-40:], dst[:40]], 1).contiguous()
    mxq.moe_scatter_quant_mxfp4(xf[-40:], src, rows, q=qf, scales=sf)
    for at in (qf[-40:], qf[:40]):
        assert torch.equal(at, q[-40:])
    for at in (sf[-40:], sf[:40]):
        assert torch.equal(at, s[-40:])
    assert bool((qf[40:-40] == 0xA5).all())


def test_balance_of_rows_far_apart():
    T, E, K = 33000, 8, 2
    say("far", T, E)
    g = torch.Generator().manual_seed(4)
    logits = torch.randn((T, E), generator=g).to(DEV)
    ids = mxq.moe_route(logits, K)[0]
    lf, gf = far(T, E, torch.float32), far(T, E, torch.float32)
    lf.copy_(logits)
    a = mxq.moe_balance_loss(logits, ids, z_loss=True)
    b = mxq.moe_balance_loss(lf, ids, z_loss=True)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    one = torch.full((1,), float(T), device=DEV)
    assert torch.equal(
        mxq.moe_balance_loss_backward(one, logits, a["counts"], grad_z=one),
        mxq.moe_balance_loss_backward(one, lf, a["counts"], grad_z=one,
                                      grad_logits=gf))
