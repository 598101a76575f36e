"""moe_expert_matmul and moe_expert_matmul_quant against the 64-bit
reference.  Payloads of two neighbouring exponents and scales of three make
products within 12 bits of each other, which the matrix unit keeps whole, and
sums that fp32 holds exactly: there the result has to be the reference's, bit
for bit.  Elsewhere the tolerance is the reference's bound of what the matrix
unit drops, plus half a step of the output's type."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import operator_refs as ref
from gpu_util import (DEV, bf16_to_host, f32_to_dev, host, i32_to_dev, say,
                      u8_to_dev)

pytestmark = pytest.mark.gpu

GROUP = {"ue8m0_g128": 128, "e8m0_g32": 32}
# hints that reach every kernel, whatever the rows really are: few rows,
# 128-row tiles (any hint a handful of tiles fits), 256-row tiles
HINTS = (1, 13, 200, 1 << 20)


class Problem:
    """Experts' rows with some padding behind each, NaN bytes and scale 255
    in the rows that no one may read into a live result."""

    def __init__(self, seed, counts, N, H, fmt, act="none", bias=False,
                 residual=False, pad=5, exact=False):
        rng = np.random.default_rng(seed)
        self.fmt, self.G, self.act = fmt, GROUP[fmt], act
        E = len(counts)
        self.E, self.N, self.H = E, N, H
        self.cols = N // 2 if act == "silu_mul" else N
        self.counts = np.asarray(counts, np.int32)
        size = self.counts + pad
        self.offsets = np.concatenate([[0], np.cumsum(size)]).astype(np.int32)
        self.rows = int(self.offsets[-1]) + 3
        q, s = self.bytes_of(rng, (self.rows, H), exact), None
        lo, hi = (126, 129) if exact else (118, 126)
        s = rng.integers(lo, hi, (self.rows, H // self.G), np.uint8)
        live = np.zeros(self.rows, bool)
        for e in range(E):
            live[self.offsets[e]:self.offsets[e] + self.counts[e]] = True
        q[~live], s[~live] = 0x7F, 255
        self.live = live
        self.q, self.s = q, s
        self.w = self.bytes_of(rng, (E, N, H), exact)
        lo, hi = (126, 129) if exact else (116, 122)
        self.ws = rng.integers(lo, hi, (E, -(-N // 128), -(-H // 128)),
                               np.uint8)
        self.bias = None
        if bias:
            b = rng.integers(-8, 9, (E, N)) if exact else \
                rng.standard_normal((E, N))
            self.bias = b.astype(np.float32)
        self.res = None
        if residual:
            r = rng.integers(-8, 9, (self.rows, self.cols)) if exact else \
                rng.standard_normal((self.rows, self.cols))
            self.res = torch.from_numpy(r.astype(np.float32)).bfloat16()

    @staticmethod
    def bytes_of(rng, shape, exact):
        # exact: 1 to 3.75, products of 6 fraction bits
        e = rng.integers(7, 9, shape, np.uint8) if exact else \
            rng.integers(3, 10, shape, np.uint8)
        m = rng.integers(0, 8, shape, np.uint8)
        sign = rng.integers(0, 2, shape, np.uint8)
        return (sign << 7) | (e << 3) | m

    def dev(self):
        return dict(q=u8_to_dev(self.q), scales=u8_to_dev(self.s),
                    w=u8_to_dev(self.w), w_scales=u8_to_dev(self.ws),
                    expert_offsets=i32_to_dev(self.offsets),
                    counts=i32_to_dev(self.counts), fmt=self.fmt,
                    act=self.act,
                    bias=None if self.bias is None else f32_to_dev(self.bias))

    def want(self):
        return ref.expert_matmul(
            self.q, self.s, self.G, self.w, self.ws, self.offsets,
            self.counts, self.bias, self.act,
            None if self.res is None else self.res.double().numpy(),
            self.cols)


def check_bf16(p, hints=HINTS, exact=False):
    d = p.dev()
    y, err = p.want()
    for hint in hints:
        out = torch.full((p.rows, p.cols), 5.0, dtype=torch.bfloat16,
                         device=DEV)
        mxq.moe_expert_matmul(
            **d, residual=None if p.res is None else p.res.to(DEV), out=out,
            expected_m=hint)
        got = out.cpu().double().numpy()
        assert (got[~p.live] == 5.0).all(), hint
        if exact:
            bad = got[p.live] != ref.bf16(y[p.live])
            assert not bad.any(), (hint, int(bad.sum()),
                                   np.argwhere(bad)[:4].tolist())
        else:
            off = np.abs(got[p.live] - y[p.live])
            lim = 2.0 ** -8 * (np.abs(y[p.live]) + err[p.live]) + err[p.live]
            assert (off <= lim + 1e-38).all(), (hint, (off / lim).max())


def check_quant(p, out_fmt, hints=HINTS):
    d = p.dev()
    y, err = p.want()
    G = GROUP[out_fmt]
    for hint in hints:
        qo = torch.full((p.rows, p.cols), 0xA5, dtype=torch.uint8, device=DEV)
        so = torch.full((p.rows, p.cols // G), 0xA5, dtype=torch.uint8,
                        device=DEV)
        mxq.moe_expert_matmul_quant(**d, out_fmt=out_fmt, q_out=qo,
                                    scales_out=so, expected_m=hint)
        gq, gs = host(qo), host(so)
        assert (gq[~p.live] == 0xA5).all() and (gs[~p.live] == 0xA5).all()
        ref.check_quantized(y, err, gq, gs, G, p.live)


COUNTS = {"one": [1], "few": [0, 3, 1, 0, 16], "odd": [17, 0, 33, 5],
          "mid": [64, 65, 0, 130], "many": [300, 1, 257]}


@pytest.mark.parametrize("fmt", ["ue8m0_g128", "e8m0_g32"])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("N,H", [(64, 128), (256, 512), (400, 640),
                                 (16, 1152), (784, 256)])
def test_exact_sums(counts, N, H, fmt, act):
    """Every product and sum is exact in fp32 (the gated form is compared
    within the reference's bound)."""
    p = Problem(N + H, COUNTS[counts], N, H, fmt, act, bias=True,
                residual=True, exact=True)
    say("exact sums", counts, N, H, fmt, act)
    check_bf16(p, exact=act == "none")


@pytest.mark.parametrize("H", [32, 64, 96, 160, 224, 672, 1376])
def test_rows_that_end_inside_a_step(H):
    p = Problem(H, [5, 0, 70, 20], 136, H, "e8m0_g32", exact=True)
    say("tail", H)
    check_bf16(p, exact=True)
    check_bf16(Problem(H, [5, 0, 70, 20], 272, H, "e8m0_g32", "silu_mul",
                       bias=True))


@pytest.mark.parametrize("fmt", ["ue8m0_g128", "e8m0_g32"])
@pytest.mark.parametrize("act,bias,residual", [
    ("none", False, False), ("none", True, True), ("silu", True, False),
    ("silu_mul", False, False), ("silu_mul", True, True)])
@pytest.mark.parametrize("counts", ["one", "odd", "many"])
def test_values(counts, act, bias, residual, fmt):
    p = Problem(11, COUNTS[counts], 528, 1024, fmt, act, bias, residual)
    say("values", counts, act, bias, residual, fmt)
    check_bf16(p)


@pytest.mark.parametrize("fmt", ["ue8m0_g128", "e8m0_g32"])
@pytest.mark.parametrize("out_fmt", ["ue8m0_g128", "e8m0_g32"])
@pytest.mark.parametrize("act", ["none", "silu", "silu_mul"])
@pytest.mark.parametrize("counts,cols", [("one", 128), ("odd", 384),
                                         ("many", 640)])
def test_quantized(counts, cols, act, out_fmt, fmt):
    N = cols * 2 if act == "silu_mul" else cols
    p = Problem(13, COUNTS[counts], N, 896, fmt, act, bias=True)
    say("quantized", counts, cols, act, out_fmt, fmt)
    check_quant(p, out_fmt)


def test_quantized_groups_of_32_past_a_block():
    for act in ("none", "silu_mul"):
        cols = 352
        N = cols * 2 if act == "silu_mul" else cols
        check_quant(Problem(17, [9, 40, 131], N, 416, "e8m0_g32", act),
                    "e8m0_g32")


def test_quantized_zero_rows_and_large_values():
    """A row of zeros gets the smallest exponent and zero payload; products
    near the ends of the exponent's range keep the rule."""
    p = Problem(19, [4, 6], 128, 256, "ue8m0_g128")
    p.q[0] = 0
    p.s[1], p.s[2] = 200, 5
    p.ws[:] = 127
    p.s[5] = 0
    check_quant(p, "ue8m0_g128")
    check_quant(p, "e8m0_g32")
    d = p.dev()
    qo, so = mxq.moe_expert_matmul_quant(**d)
    assert (host(qo)[0] & 0x7F == 0).all() and (host(so)[0] == 0).all()


@pytest.mark.parametrize("hint", HINTS)
def test_device_data_out_of_range(hint):
    """Counts and offsets that no layout makes: nothing outside the rows is
    read or written."""
    p = Problem(23, [10, 10, 10, 10], 256, 256, "ue8m0_g128")
    d = p.dev()
    y, err = p.want()
    end = p.rows
    cases = [([-5, 10, 3, 1 << 30], p.offsets),
             ([10, 10, 10, 10], np.array([0, 15, 30, 45, 1 << 30])),
             ([10, 10, 10, 10], np.array([-8, 15, 30, end, end + 60])),
             ([10, 10, 10, 10], np.array([40, 15, end + 7, 45, 30]))]
    for counts, offsets in cases:
        out = torch.full((p.rows + 4, p.cols), 5.0, dtype=torch.bfloat16,
                         device=DEV)
        d["counts"] = i32_to_dev(counts)
        d["expert_offsets"] = i32_to_dev(offsets)
        mxq.moe_expert_matmul(**d, out=out, expected_m=hint)
        got = out.cpu().double().numpy()
        assert (got[p.rows:] == 5).all()
        live = np.zeros(p.rows + 4, bool)
        for e in range(4):
            a, n = ref.live_rows(offsets, counts, p.rows, e)
            live[a:a + n] = n > 0
        assert (got[~live] == 5).all()


@pytest.mark.parametrize("hint", HINTS)
def test_strides(hint):
    p = Problem(29, [20, 3, 150], 272, 384, "e8m0_g32", "silu_mul",
                residual=True)
    d = p.dev()
    res = p.res.to(DEV)
    plain = torch.zeros((p.rows, p.cols), dtype=torch.bfloat16, device=DEV)
    mxq.moe_expert_matmul(**d, residual=res, out=plain, expected_m=hint)

    def wide(t, left, right):
        big = torch.full((t.shape[0], left + t.shape[1] + right), 0x7F,
                         dtype=t.dtype, device=DEV)
        v = big[:, left:left + t.shape[1]]
        v.copy_(t)
        return v, big

    d["q"], _ = wide(d["q"], 16, 32)
    d["scales"], _ = wide(d["scales"], 3, 2)
    res, _ = wide(res, 8, 8)
    out, big = wide(torch.zeros_like(plain), 8, 16)
    mxq.moe_expert_matmul(**d, residual=res, out=out, expected_m=hint)
    assert torch.equal(out, plain)
    assert (big[:, :8] == 0x7F).all() and (big[:, 8 + p.cols:] == 0x7F).all()
    # in place over the residual
    mxq.moe_expert_matmul(**d, residual=res, out=res, expected_m=hint)
    live = torch.from_numpy(p.live).to(DEV)
    assert torch.equal(res[live], plain[live])
    # quantized output into wider rows
    p = Problem(31, [20, 3, 150], 256, 384, "e8m0_g32")
    d = p.dev()
    a, b = mxq.moe_expert_matmul_quant(**{**d, "act": "none"},
                                       expected_m=hint)
    qo = torch.full((p.rows, 256 + 32), 0xA5, dtype=torch.uint8, device=DEV)
    so = torch.full((p.rows, 2 + 3), 0xA5, dtype=torch.uint8, device=DEV)
    mxq.moe_expert_matmul_quant(**{**d, "act": "none"}, q_out=qo[:, 16:272],
                                scales_out=so[:, 1:3], expected_m=hint)
    live = torch.from_numpy(p.live).to(DEV)
    assert torch.equal(qo[:, 16:272][live], a[live])
    assert torch.equal(so[:, 1:3][live], b[live])
    assert (qo[:, :16] == 0xA5).all() and (qo[:, 272:] == 0xA5).all()
    assert (so[:, 0] == 0xA5).all() and (so[:, 3:] == 0xA5).all()


@pytest.mark.parametrize("act,N", [("none", 132), ("none", 4),
                                   ("silu_mul", 1432), ("silu_mul", 264)])
def test_rows_on_8_bytes(act, N):
    """Columns and strides that are multiples of four."""
    p = Problem(59, [20, 3, 140], N, 352, "e8m0_g32", act, bias=True,
                residual=True, exact=act == "none")
    check_bf16(p, exact=act == "none")
    d = p.dev()
    out = torch.full((p.rows, p.cols + 8), 5.0, dtype=torch.bfloat16,
                     device=DEV)
    for hint in HINTS:
        plain = mxq.moe_expert_matmul(**d, expected_m=hint)
        mxq.moe_expert_matmul(**d, out=out[:, 4:4 + p.cols], expected_m=hint)
        live = torch.from_numpy(p.live).to(DEV)
        assert torch.equal(out[:, 4:4 + p.cols][live], plain[live])
        assert (out[:, :4] == 5).all() and (out[:, 4 + p.cols:] == 5).all()


def test_nan_bytes_stay_in_their_rows():
    p = Problem(37, [20, 130], 128, 256, "ue8m0_g128")
    p.q[3, 17] = 0x7F          # live row 3 of expert 0
    d = p.dev()
    for hint in HINTS:
        out = mxq.moe_expert_matmul(**d, expected_m=hint).cpu()
        live = torch.from_numpy(p.live)
        nan = torch.isnan(out).any(1) & live
        assert nan.nonzero().flatten().tolist() == [3]
        assert torch.isnan(out[3]).all()


def test_shapes_at_the_ends():
    # no rows at all
    p = Problem(41, [0, 0], 64, 128, "ue8m0_g128", pad=0)
    d = p.dev()
    out = torch.full((p.rows, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    mxq.moe_expert_matmul(**d, out=out)
    assert (out == 5).all()
    d["q"], d["scales"] = d["q"][:0], d["scales"][:0]
    assert mxq.moe_expert_matmul(**d).shape == (0, 64)
    # the smallest product, and the most experts
    check_bf16(Problem(43, [1], 8, 32, "e8m0_g32", exact=True), exact=True)
    counts = [(i * 7) % 4 for i in range(1024)]
    check_bf16(Problem(47, counts, 8, 32, "e8m0_g32", pad=1, exact=True),
               exact=True)


def test_refusals():
    p = Problem(53, [4, 6], 128, 256, "ue8m0_g128")
    d = p.dev()

    def call(quant=False, **kw):
        a = {**d, **kw}
        if quant:
            return mxq.moe_expert_matmul_quant(**a)
        return mxq.moe_expert_matmul(**a)

    for kw in (dict(w=d["w"][:, :, :128].contiguous()),
               dict(w_scales=d["w_scales"][:, :, :1].contiguous()),
               dict(counts=d["counts"][:1]),
               dict(counts=d["counts"].long()),
               dict(expert_offsets=d["expert_offsets"][:2]),
               dict(scales=d["scales"][:, :1]),
               dict(scales=d["scales"][:3]),
               dict(bias=torch.zeros((2, 127), device=DEV)),
               dict(residual=torch.zeros((p.rows, 127), device=DEV,
                                         dtype=torch.bfloat16)),
               dict(out=torch.zeros((p.rows - 1, 128), device=DEV,
                                    dtype=torch.bfloat16)),
               dict(w=d["w"].cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(q=d["q"].float()), dict(scales=d["scales"].int()),
               dict(out=torch.zeros((p.rows, 128), device=DEV)),
               dict(residual=torch.zeros((p.rows, 128), device=DEV))):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(KeyError):
        call(act="relu")
    with pytest.raises(KeyError):
        call(fmt="ue4m3")
    with pytest.raises(mxq.MxqError):
        call(expected_m=-1)
    with pytest.raises(mxq.MxqError):   # rows that start off 8 bytes
        call(out=torch.zeros((p.rows, 132), device=DEV,
                             dtype=torch.bfloat16)[:, 2:130])
    with pytest.raises(mxq.MxqError):   # 66 gated columns
        call(act="silu_mul", w=torch.zeros((2, 132, 256), device=DEV,
                                           dtype=torch.uint8),
             w_scales=torch.zeros((2, 2, 2), device=DEV, dtype=torch.uint8))
    # 64 gated columns hold no group of 128
    with pytest.raises(mxq.MxqError):
        call(quant=True, act="silu_mul")


@pytest.mark.parametrize("hint", HINTS)
def test_rows_far_apart(hint):
    """Rows, scales, residual and output beyond 2^32 bytes of their starts:
    the widest row strides the call takes."""
    p = Problem(61, [20, 300], 128, 256, "ue8m0_g128", residual=True,
                exact=True)
    d = p.dev()
    res = p.res.to(DEV)
    plain = mxq.moe_expert_matmul(**d, residual=res, expected_m=hint)
    rows, ld, at = 1400, 1 << 22, 1060  # expert 1 begins past 2^32 bytes
    a, b = int(p.offsets[1]), int(p.counts[1])
    src = torch.cat([torch.arange(20), torch.arange(a, a + b)]).to(DEV)
    dst = torch.cat([torch.arange(20), torch.arange(at, at + b)]).to(DEV)

    def far(t):
        big = torch.empty((rows, ld // t.element_size()), dtype=t.dtype,
                          device=DEV)[:, :t.shape[1]]
        big[dst] = t[src]
        return big

    say("rows far apart", hint)
    d["q"], d["scales"], res = far(d["q"]), far(d["scales"]), far(res)
    d["expert_offsets"] = i32_to_dev([0, at, at + b])
    out = far(torch.zeros_like(plain))
    mxq.moe_expert_matmul(**d, residual=res, out=out, expected_m=hint)
    assert torch.equal(out[dst], plain[src])
