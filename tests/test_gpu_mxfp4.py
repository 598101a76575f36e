"""Quantization to microscaled 4-bit floats and back, bit for bit against the
64-bit reference."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import mx_refs as mx
import operator_refs as ref
from gpu_util import DEV, assert_equal, host, i32_to_dev, say, u8_to_dev

pytestmark = pytest.mark.gpu
C = 0xA5
RULES = ("no_clip", "ocp_floor")


def values(seed, rows, H, dtype):
    """Rows of their own size, with zeros, zero groups and halfway values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, H), generator=g) * torch.exp(
        3 * torch.randn((rows, 1), generator=g))
    x[:, ::37] = 0
    x[rows // 2, :32] = 0
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x[rows - 1, -32:] = torch.cat([half, -half, half / 2, -half])
    return x.to(dtype).to(DEV)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H", [(1, 32), (3, 64), (300, 32), (129, 96),
                                    (33, 1376), (17, 7168), (5, 8224),
                                    (2, 33024), (1, 131072), (1000, 352)])
def test_rows(rows, H, dtype, rule):
    say("mxfp4 rows", rows, H, dtype, rule)
    x = values(rows + H, rows, H, dtype)
    q, s = mxq.mxfp4_quant_rows(x, rule)
    wq, ws = mx.quant(x.double().cpu().numpy(), rule)
    assert_equal(host(q), wq, "payload")
    assert_equal(host(s), ws, "scales")


@pytest.mark.parametrize("rule", RULES)
def test_extreme_values(rule):
    """Every finite bf16 value in groups of its own size and beside others,
    subnormal fp32, the largest fp32."""
    v = (torch.arange(65536, dtype=torch.int32) << 16).view(torch.float32)
    v = v[torch.isfinite(v)]
    v = torch.cat([v, torch.zeros(-v.numel() % 32)])
    for x in (v.reshape(-1, 32), v.reshape(32, -1).t().contiguous(),
              v.reshape(-1, 32) * 2.0 ** -20):
        q, s = mxq.mxfp4_quant_rows(x.to(DEV), rule)
        wq, ws = mx.quant(x.double().numpy(), rule)
        assert_equal(host(s), ws, "scales")
        assert_equal(host(q), wq, "payload")
    x = torch.full((2, 32), 3.402823466e38)
    x[1] = 1e-44
    q, s = mxq.mxfp4_quant_rows(x.to(DEV), rule)
    wq, ws = mx.quant(x.double().numpy(), rule)
    assert_equal(host(q), wq, "ends, payload")
    assert_equal(host(s), ws, "ends, scales")


def test_borders_between_codes_and_exponents():
    """fp32 values next to every halfway point and every exponent border."""
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x = torch.cat([torch.nextafter(half, torch.tensor(0.0)), half,
                   torch.nextafter(half, torch.tensor(9.0)),
                   torch.full((8,), 6.0)]).reshape(1, 32)
    rows = [x]
    for top in (3.0, 4.0, 6.0, 8.0):
        for t in (torch.tensor(0.0), torch.tensor(9.0), None):
            y = x.clone().clamp(max=2.9)
            y[0, 31] = top if t is None else torch.nextafter(
                torch.tensor(top), t)
            rows.append(y)
    x = torch.cat(rows)
    x = torch.cat([x, x * 2.0 ** -100, x * 2.0 ** 90])
    for rule in RULES:
        q, s = mxq.mxfp4_quant_rows(x.to(DEV), rule)
        wq, ws = mx.quant(x.double().numpy(), rule)
        assert_equal(host(s), ws, "scales")
        assert_equal(host(q), wq, "payload")


def test_strides_and_weights():
    x = values(1, 40, 160, torch.bfloat16)
    q, s = mxq.mxfp4_quant_rows(x)
    big = torch.zeros((40, 8 + 160 + 16), dtype=torch.bfloat16, device=DEV)
    big[:, 8:168] = x
    qo = torch.full((40, 16 + 80 + 16), C, dtype=torch.uint8, device=DEV)
    so = torch.full((40, 3 + 5 + 1), C, dtype=torch.uint8, device=DEV)
    mxq.mxfp4_quant_rows(big[:, 8:168], q=qo[:, 16:96], scales=so[:, 3:8])
    assert torch.equal(qo[:, 16:96], q) and torch.equal(so[:, 3:8], s)
    assert (qo[:, :16] == C).all() and (qo[:, 96:] == C).all()
    assert (so[:, :3] == C).all() and (so[:, 8:] == C).all()
    # weights: three dimensions, scale rows that start on 16 bytes
    w = x.reshape(4, 10, 160)
    q3, s3 = mxq.mxfp4_quant_rows(w)
    assert q3.shape == (4, 10, 80) and s3.shape == (4, 10, 5)
    assert s3.stride(1) % 16 == 0
    assert torch.equal(q3.reshape(40, 80), q)
    assert torch.equal(s3.reshape(40, 5), s)
    with pytest.raises(ValueError):
        mxq.mxfp4_quant_rows(x.reshape(4, 10, 160)[:, :9])
    # no rows
    q, s = mxq.mxfp4_quant_rows(x[:0])
    assert q.shape == (0, 80) and s.shape == (0, 5)


def test_all_bytes_back():
    """Every byte widened to e4m3 and, under every scale byte, to bf16."""
    q = torch.arange(256, dtype=torch.uint8).reshape(1, 256)
    want = mx.E2M1[mx.unpack(q.numpy())]
    out = mxq.mxfp4_to_e4m3(q.to(DEV))
    assert np.array_equal(ref.E4M3[host(out)], want)
    assert np.array_equal(np.signbit(ref.E4M3[host(out)]), np.signbit(want))
    q = q.expand(256, 256).contiguous().to(DEV)
    s = torch.arange(256, dtype=torch.uint8).reshape(256, 1).expand(256, 16)
    out = mxq.upscale_mxfp4_to_bf16(q, s.contiguous().to(DEV))
    f = np.ldexp(np.ones((256, 1)), np.arange(256)[:, None] - 127)
    v = np.broadcast_to(want, (256, 512)) * f
    v[255] = np.nan
    got = out.double().cpu().numpy()
    with np.errstate(over="ignore"):
        v = np.where(np.abs(v) > 3.4e38, np.copysign(np.inf, v), v)
    assert np.array_equal(got, v, equal_nan=True)


@pytest.mark.parametrize("rows,H", [(1, 32), (300, 96), (33, 1376),
                                    (17, 7168), (2, 33024)])
def test_back(rows, H):
    rng = np.random.default_rng(H)
    q = rng.integers(0, 256, (rows, H // 2), np.uint8)
    s = rng.integers(90, 160, (rows, H // 32), np.uint8)
    say("mxfp4 back", rows, H)
    got = mxq.upscale_mxfp4_to_bf16(u8_to_dev(q), u8_to_dev(s))
    assert np.array_equal(got.double().cpu().numpy(),
                          mx.values(q, s, "mxfp4"))
    wide = mxq.mxfp4_to_e4m3(u8_to_dev(q))
    assert np.array_equal(ref.E4M3[host(wide)], mx.E2M1[mx.unpack(q)])
    # fewer rows, wider buffers
    n = rows // 2
    out = torch.full((rows, H + 16), 5.0, dtype=torch.bfloat16, device=DEV)
    mxq.upscale_mxfp4_to_bf16(u8_to_dev(q), u8_to_dev(s), n,
                              out=out[:, 8:8 + H])
    assert torch.equal(out[:n, 8:8 + H], got[:n])
    assert (out[n:] == 5).all() and (out[:, :8] == 5).all()
    out = torch.full((rows + 1, H + 32), C, dtype=torch.uint8, device=DEV)
    mxq.mxfp4_to_e4m3(u8_to_dev(q), out=out[:, 16:16 + H])
    assert torch.equal(out[:rows, 16:16 + H], wide)
    assert (out[rows:] == C).all() and (out[:, :16] == C).all()


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("T,K,E,H,kind", [
    (1, 1, 1, 32, "compact"), (5, 3, 8, 96, "compact"),
    (64, 8, 16, 1376, "masked"), (33, 2, 4, 7168, "compact"),
    (9, 20, 40, 352, "compact"), (3, 64, 64, 32768, "compact"),
    (200, 4, 32, 640, "masked")])
def test_scatter(T, K, E, H, kind, rule):
    x = values(T + H, T, H, torch.bfloat16)
    g = torch.Generator().manual_seed(T)
    ids = torch.rand((T, E), generator=g).topk(K, 1).indices.int()
    ids[::3, 0] = -1
    lay = mxq.moe_layout(ids.to(DEV), 0, E, kind, capacity=16)
    R = lay["num_rows"]
    q = torch.full((R, H // 2), C, dtype=torch.uint8, device=DEV)
    s = torch.full((R, H // 32), C, dtype=torch.uint8, device=DEV)
    say("mxfp4 scatter", T, K, E, H, kind, rule)
    mxq.moe_scatter_quant_mxfp4(x, lay["src2dst"], R, rule, q, s)
    wq, ws = mx.quant(x.double().cpu().numpy(), rule)
    rq = np.full((R, H // 2), C, np.uint8)
    rs = np.full((R, H // 32), C, np.uint8)
    src = host(lay["src2dst"])
    for t in range(T):
        for d in src[t]:
            if d >= 0:
                rq[d], rs[d] = wq[t], ws[t]
    assert_equal(host(q), rq, "payload")
    assert_equal(host(s), rs, "scales")


def test_scatter_destinations_out_of_range_and_strides():
    x = values(3, 6, 96, torch.bfloat16)
    src = i32_to_dev([[0, -1], [9, 1], [10, 1 << 30], [-7, 2], [3, 4], [5, 6]])
    q = torch.full((12, 16 + 48 + 16), C, dtype=torch.uint8, device=DEV)
    s = torch.full((12, 2 + 3 + 1), C, dtype=torch.uint8, device=DEV)
    big = torch.zeros((6, 8 + 96 + 8), dtype=torch.bfloat16, device=DEV)
    big[:, 8:104] = x
    mxq.moe_scatter_quant_mxfp4(big[:, 8:104], src, 10, q=q[:, 16:64],
                                scales=s[:, 2:5])
    wq, ws = mx.quant(x.double().cpu().numpy())
    rq, rs = np.full((12, 80), C, np.uint8), np.full((12, 6), C, np.uint8)
    for t, row in enumerate(host(src)):
        for d in row:
            if 0 <= d < 10:
                rq[d, 16:64], rs[d, 2:5] = wq[t], ws[t]
    assert_equal(host(q), rq, "payload")
    assert_equal(host(s), rs, "scales")
    # nothing to do
    mxq.moe_scatter_quant_mxfp4(x[:0], src[:0], 10)
    mxq.moe_scatter_quant_mxfp4(x, src[:, :0], 10)


def test_graph():
    x = values(5, 40, 352, torch.bfloat16)
    src = i32_to_dev(np.arange(80).reshape(40, 2))
    side = torch.cuda.Stream()

    def step():
        q, s = mxq.moe_scatter_quant_mxfp4(x, src, 80)
        a = mxq.mxfp4_to_e4m3(q)
        b = mxq.upscale_mxfp4_to_bf16(q, s)
        return (q, s, a, b) + mxq.mxfp4_quant_rows(x, "ocp_floor")

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(values(50 + i, 40, 352, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_refusals():
    x = values(7, 8, 64, torch.bfloat16)
    q, s = mxq.mxfp4_quant_rows(x)
    src = i32_to_dev(np.arange(8).reshape(8, 1))
    for f in (lambda: mxq.mxfp4_quant_rows(x.cpu()),
              lambda: mxq.mxfp4_quant_rows(x, q=q[:4]),
              lambda: mxq.mxfp4_quant_rows(x, scales=s[:, :1]),
              lambda: mxq.mxfp4_quant_rows(x, q=q.cpu()),
              lambda: mxq.moe_scatter_quant_mxfp4(x, src[:4], 8),
              lambda: mxq.moe_scatter_quant_mxfp4(x, src, 8, q=q[:7]),
              lambda: mxq.mxfp4_to_e4m3(q, out=q),
              lambda: mxq.upscale_mxfp4_to_bf16(q, s[:7]),
              lambda: mxq.upscale_mxfp4_to_bf16(q, s, 9)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        mxq.mxfp4_quant_rows(x.half())
    with pytest.raises(TypeError):
        mxq.moe_scatter_quant_mxfp4(x.float(), src, 8)
    with pytest.raises(KeyError):
        mxq.mxfp4_quant_rows(x, "nearest")
    with pytest.raises(mxq.MxqError):   # 48 channels hold no whole groups
        mxq.mxfp4_quant_rows(x[:, :48])
    with pytest.raises(mxq.MxqError):   # rows that start off 16 bytes
        mxq.mxfp4_quant_rows(torch.zeros((4, 72), dtype=torch.bfloat16,
                                         device=DEV)[:, 4:68])
    # 4-bit rows are no format of the 8-bit calls
    with pytest.raises(KeyError):
        mxq.moe_scatter_quant(x, src, 8, fmt="mxfp4")
