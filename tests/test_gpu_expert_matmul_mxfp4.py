"""moe_expert_matmul_mxfp4 and moe_expert_matmul_mxfp4_quant against the
64-bit reference.  Products of e2m1 payloads are multiples of 1/4 up to 36,
and with scales of one and two all sums here are whole multiples of 1/4 far
below 2^24 of them, which fp32 holds: there the result has to be the
reference's, bit for bit.  So too with e4m3 rows between 1 and 3.75, whose
products with e2m1 lie within 13 bits of each other.  Elsewhere the tolerance
is the reference's bound plus half a step of the output's type."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import mx_refs as mx
import operator_refs as ref
from gpu_util import DEV, f32_to_dev, host, i32_to_dev, say, u8_to_dev

pytestmark = pytest.mark.gpu

FMTS = ("mxfp4", "e8m0_g32")
# hints that reach every kernel of few blocks, whatever the rows really are,
# and those of many
HINTS = (1, 13, 40, 200, 1 << 20)
MANY_HINTS = (1, 7, 13, 18)


class Problem:
    """Experts' rows with some padding behind each, NaN bytes (e4m3) and scale
    255 in the rows that no one may read into a live result."""

    def __init__(self, seed, counts, N, H, fmt, act="none", bias=False,
                 residual=False, pad=5, exact=False):
        rng = np.random.default_rng(seed)
        self.fmt, self.act = fmt, act
        E = len(counts)
        self.E, self.N, self.H = E, N, H
        self.cols = N // 2 if act == "silu_mul" else N
        self.counts = np.asarray(counts, np.int32)
        self.offsets = np.concatenate(
            [[0], np.cumsum(self.counts + pad)]).astype(np.int32)
        self.rows = int(self.offsets[-1]) + 3
        live = np.zeros(self.rows, bool)
        for e in range(E):
            live[self.offsets[e]:self.offsets[e] + self.counts[e]] = True
        self.live = live
        if fmt == "mxfp4":
            q = rng.integers(0, 256, (self.rows, H // 2), np.uint8)
        else:
            e = rng.integers(7, 9, (self.rows, H), np.uint8) if exact else \
                rng.integers(3, 10, (self.rows, H), np.uint8)
            q = (rng.integers(0, 2, e.shape, np.uint8) << 7) | (e << 3) | \
                rng.integers(0, 8, e.shape, np.uint8)
        lo, hi = (127, 129) if exact else (118, 126)
        s = rng.integers(lo, hi, (self.rows, H // 32), np.uint8)
        q[~live], s[~live] = 0x7F, 255
        self.q, self.s = q, s
        self.w = rng.integers(0, 256, (E, N, H // 2), np.uint8)
        lo, hi = (127, 129) if exact else (117, 124)
        # rows of scales start on 4 bytes; what is behind them is NaN
        self.ld = -(-(H // 32) // 4) * 4
        self.ws = np.full((E, N, self.ld), 255, np.uint8)
        self.ws[:, :, :H // 32] = rng.integers(lo, hi, (E, N, H // 32),
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

    def dev(self):
        return dict(q=u8_to_dev(self.q), scales=u8_to_dev(self.s),
                    w=u8_to_dev(self.w),
                    w_scales=u8_to_dev(self.ws)[:, :, :self.H // 32],
                    expert_offsets=i32_to_dev(self.offsets),
                    counts=i32_to_dev(self.counts), fmt=self.fmt,
                    act=self.act,
                    bias=None if self.bias is None else f32_to_dev(self.bias))

    def want(self):
        return mx.expert_matmul(
            self.q, self.s, self.fmt, self.w, self.ws[:, :, :self.H // 32],
            self.offsets, self.counts, self.bias, self.act,
            None if self.res is None else self.res.double().numpy(),
            self.cols)


def check_bf16(p, hints=HINTS, exact=False):
    d = p.dev()
    y, err = p.want()
    for hint in hints:
        out = torch.full((p.rows, p.cols), 5.0, dtype=torch.bfloat16,
                         device=DEV)
        mxq.moe_expert_matmul_mxfp4(
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
    pay = p.cols // 2 if out_fmt == "mxfp4" else p.cols
    for hint in hints:
        qo = torch.full((p.rows, -(-pay // 16) * 16), 0xA5,
                        dtype=torch.uint8, device=DEV)[:, :pay]
        so = torch.full((p.rows, p.cols // 32), 0xA5, dtype=torch.uint8,
                        device=DEV)
        mxq.moe_expert_matmul_mxfp4_quant(**d, out_fmt=out_fmt, q_out=qo,
                                          scales_out=so, expected_m=hint)
        gq, gs = host(qo), host(so)
        assert (gq[~p.live] == 0xA5).all() and (gs[~p.live] == 0xA5).all()
        if out_fmt == "mxfp4":
            mx.check_quantized(y, err, gq, gs, p.live)
        else:
            ref.check_quantized(y, err, gq, gs, 32, p.live)


COUNTS = {"one": [1], "few": [0, 3, 1, 0, 16], "odd": [17, 0, 33, 5],
          "mid": [64, 65, 0, 130], "many": [300, 1, 257]}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("N,H", [(64, 128), (256, 512), (400, 640),
                                 (16, 1152), (784, 256)])
def test_exact_sums(counts, N, H, fmt, act):
    p = Problem(N + H, COUNTS[counts], N, H, fmt, act, bias=True,
                residual=True, exact=True)
    say("mxfp4 exact sums", counts, N, H, fmt, act)
    check_bf16(p, exact=act == "none")


# 140 experts: more blocks than CUs, of 128 weight rows and of 256
MANY = [(0, 1, 16, 17, 3, 33, 48, 49, 0, 64, 65, 2)[i % 12]
        for i in range(140)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("N,H", [(272, 32), (400, 224), (520, 512),
                                 (264, 1056)])
def test_many_blocks(N, H, act, fmt):
    p = Problem(N + H, MANY, N, H, fmt, act, bias=True, residual=True, pad=2,
                exact=True)
    say("mxfp4 many blocks", N, H, act, fmt)
    check_bf16(p, MANY_HINTS, exact=act == "none")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_fmt", FMTS)
@pytest.mark.parametrize("act,N", [("none", 288), ("silu_mul", 576)])
def test_many_blocks_quantized(act, N, out_fmt, fmt):
    say("mxfp4 many blocks, quantized", act, N, out_fmt, fmt)
    check_quant(Problem(3, MANY, N, 416, fmt, act, bias=True, pad=1), out_fmt,
                MANY_HINTS)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hint", MANY_HINTS)
def test_many_blocks_device_data_and_strides(hint, fmt):
    """Offsets and counts that no layout makes, scales of tokens that start
    on no word, NaN of one row and one weight row."""
    p = Problem(5, MANY, 272, 352, fmt, exact=True)
    p.s[int(p.offsets[3]) + 4, 5] = 255
    p.ws[7, 200, 10] = 255
    d = p.dev()
    d["scales"], _ = wide(d["scales"], 3, 2)
    d["q"], _ = wide(d["q"], 16, 32)
    out = mxq.moe_expert_matmul_mxfp4(**d, expected_m=hint).cpu()
    nan = torch.isnan(out) & torch.from_numpy(p.live)[:, None]
    a, n = int(p.offsets[7]), int(p.counts[7])
    want = torch.zeros_like(nan)
    want[int(p.offsets[3]) + 4] = True
    want[a:a + n, 200] = True
    assert torch.equal(nan, want)
    counts, offsets = p.counts.copy(), p.offsets.copy()
    counts[0], counts[5], counts[9] = -3, 1 << 30, 1 << 30
    offsets[20] = -7
    offsets[30] = p.rows + 50
    d["counts"], d["expert_offsets"] = i32_to_dev(counts), i32_to_dev(offsets)
    out = torch.full((p.rows + 4, p.cols), 5.0, dtype=torch.bfloat16,
                     device=DEV)
    mxq.moe_expert_matmul_mxfp4(**d, out=out, expected_m=hint)
    live = np.zeros(p.rows + 4, bool)
    for e in range(p.E):
        a, n = ref.live_rows(offsets, counts, p.rows, e)
        live[a:a + n] = n > 0
    assert (out.cpu().double().numpy()[~live] == 5).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [32, 64, 96, 128, 160, 224, 288, 480, 672, 1376,
                               2080])
def test_rows_that_end_inside_a_step(H, fmt):
    say("mxfp4 tail", H, fmt)
    check_bf16(Problem(H, [5, 0, 70, 20], 136, H, fmt, exact=True),
               exact=True)
    check_bf16(Problem(H, [5, 0, 70, 20], 272, H, fmt, "silu_mul", bias=True))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act,bias,residual", [
    ("none", False, False), ("none", True, True), ("silu", True, False),
    ("silu_mul", False, False), ("silu_mul", True, True)])
@pytest.mark.parametrize("counts", ["one", "odd", "many"])
def test_values(counts, act, bias, residual, fmt):
    say("mxfp4 values", counts, act, bias, residual, fmt)
    check_bf16(Problem(11, COUNTS[counts], 528, 1024, fmt, act, bias,
                       residual))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_fmt", FMTS)
@pytest.mark.parametrize("act", ["none", "silu", "silu_mul"])
@pytest.mark.parametrize("counts,cols", [("one", 32), ("odd", 352),
                                         ("many", 640)])
def test_quantized(counts, cols, act, out_fmt, fmt):
    N = cols * 2 if act == "silu_mul" else cols
    say("mxfp4 quantized", counts, cols, act, out_fmt, fmt)
    check_quant(Problem(13, COUNTS[counts], N, 896, fmt, act, bias=True),
                out_fmt)


def test_quantized_zero_rows_and_large_values():
    p = Problem(19, [4, 6], 128, 256, "mxfp4")
    p.q[0] = 0
    p.s[1], p.s[2], p.s[5] = 200, 5, 0
    p.ws[:, :, :8] = 127
    for out_fmt in FMTS:
        check_quant(p, out_fmt)
    qo, so = mxq.moe_expert_matmul_mxfp4_quant(**p.dev())
    assert (host(qo)[0] & 0x77 == 0).all() and (host(so)[0] == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_bytes_stay_in_their_rows(fmt):
    """A scale of 255, and in 8-bit rows a NaN byte: that row alone."""
    p = Problem(37, [20, 130], 128, 256, fmt)
    p.s[3, 5] = 255
    if fmt != "mxfp4":
        p.q[3, 17] = 0x7F
    d = p.dev()
    for hint in HINTS:
        out = mxq.moe_expert_matmul_mxfp4(**d, expected_m=hint).cpu()
        nan = torch.isnan(out).any(1) & torch.from_numpy(p.live)
        assert nan.nonzero().flatten().tolist() == [3]
        assert torch.isnan(out[3]).all()
    # and of a weight row: that column of its expert's rows
    p = Problem(38, [20, 130], 128, 256, fmt)
    p.ws[1, 77, 2] = 255
    d = p.dev()
    for hint in HINTS:
        out = mxq.moe_expert_matmul_mxfp4(**d, expected_m=hint).cpu()
        nan = torch.isnan(out) & torch.from_numpy(p.live)[:, None]
        assert nan.any(0).nonzero().flatten().tolist() == [77]
        assert int(nan.sum()) == 130


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hint", HINTS)
def test_device_data_out_of_range(hint, fmt):
    """Counts and offsets that no layout makes: nothing outside the rows is
    read or written."""
    p = Problem(23, [10, 10, 10, 10], 256, 256, fmt)
    d = p.dev()
    end = p.rows
    for counts, offsets in (
            ([-5, 10, 3, 1 << 30], p.offsets),
            ([10, 10, 10, 10], np.array([0, 15, 30, 45, 1 << 30])),
            ([10, 10, 10, 10], np.array([-8, 15, 30, end, end + 60])),
            ([10, 10, 10, 10], np.array([40, 15, end + 7, 45, 30]))):
        out = torch.full((p.rows + 4, p.cols), 5.0, dtype=torch.bfloat16,
                         device=DEV)
        d["counts"], d["expert_offsets"] = i32_to_dev(counts), \
            i32_to_dev(offsets)
        mxq.moe_expert_matmul_mxfp4(**d, out=out, expected_m=hint)
        got = out.cpu().double().numpy()
        live = np.zeros(p.rows + 4, bool)
        for e in range(4):
            a, n = ref.live_rows(offsets, counts, p.rows, e)
            live[a:a + n] = n > 0
        assert (got[~live] == 5).all()


def wide(t, left, right, fill=0x7F):
    big = torch.full((t.shape[0], left + t.shape[1] + right), fill,
                     dtype=t.dtype, device=DEV)
    v = big[:, left:left + t.shape[1]]
    v.copy_(t)
    return v, big


# rows of more than 2560 channels, and of 8 bits of more than 4096, go through
# 256-row tiles where there are many; scales in chunks of 512 channels, the last
# one whole, cut or missing
LONG = (1056, 1504, 2048, 2592, 4128, 4608, 5216)
LONG_HINTS = (13, 40, 1 << 20)  # the K split, and both sizes of tiles


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act,N", [("none", 272), ("silu_mul", 400)])
@pytest.mark.parametrize("H", LONG)
def test_long_rows(H, act, N, fmt):
    say("mxfp4 long rows", H, act, N, fmt)
    p = Problem(H, [300, 1, 0, 257, 64], N, H, fmt, act, bias=True,
                residual=act == "none", exact=True)
    check_bf16(p, LONG_HINTS, exact=act == "none")
    # scales of tokens that start on no word: the same bytes
    d = p.dev()
    for hint in LONG_HINTS:
        plain = mxq.moe_expert_matmul_mxfp4(**d, expected_m=hint)
        far, _ = wide(d["scales"], 3, 2, 0xFF)
        out = mxq.moe_expert_matmul_mxfp4(**{**d, "scales": far},
                                          expected_m=hint)
        live = torch.from_numpy(p.live).to(DEV)
        assert torch.equal(out[live], plain[live]), hint


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_fmt", FMTS)
@pytest.mark.parametrize("act,N", [("none", 288), ("silu_mul", 576)])
@pytest.mark.parametrize("H", (1120, 4192))
def test_long_rows_quantized(H, act, N, out_fmt, fmt):
    say("mxfp4 long rows, quantized", H, act, N, out_fmt, fmt)
    check_quant(Problem(6, [260, 70, 0, 1], N, H, fmt, act, bias=True, pad=1),
                out_fmt, LONG_HINTS)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", (1504, 4128))
def test_long_rows_nan_and_device_data(H, fmt):
    """A scale of 255 in the last block of one row and of one weight row, and
    offsets and counts that no layout makes."""
    p = Problem(8, [260, 70, 3], 272, H, fmt, exact=True)
    p.s[150, H // 32 - 1] = 255
    p.ws[1, 200, H // 32 - 1] = 255
    a = int(p.offsets[1])
    want = torch.zeros((p.rows, 272), dtype=torch.bool)
    want[150] = True
    want[a:a + 70, 200] = True
    for hint in LONG_HINTS:
        for wider in (False, True):
            d = p.dev()
            if wider:
                d["scales"], _ = wide(d["scales"], 3, 2, 0xFF)
            out = mxq.moe_expert_matmul_mxfp4(**d, expected_m=hint).cpu()
            nan = torch.isnan(out) & torch.from_numpy(p.live)[:, None]
            assert torch.equal(nan, want), (hint, wider)
    for counts, offsets in (
            ([-5, 1 << 30, 10], p.offsets),
            ([260, 260, 260], np.array([0, 200, 300, 1 << 30])),
            ([260, 70, 3], np.array([-8, 100, p.rows, p.rows + 60]))):
        d = p.dev()
        d["counts"], d["expert_offsets"] = i32_to_dev(counts), \
            i32_to_dev(offsets)
        live = np.zeros(p.rows + 4, bool)
        for e in range(3):
            a, n = ref.live_rows(offsets, counts, p.rows, e)
            live[a:a + n] = n > 0
        for hint in LONG_HINTS:
            out = torch.full((p.rows + 4, p.cols), 5.0, dtype=torch.bfloat16,
                             device=DEV)
            mxq.moe_expert_matmul_mxfp4(**d, out=out, expected_m=hint)
            assert (out.cpu().double().numpy()[~live] == 5).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hint", HINTS)
def test_strides(hint, fmt):
    p = Problem(29, [20, 3, 150], 272, 352, fmt, "silu_mul", residual=True)
    d = p.dev()
    res = p.res.to(DEV)
    plain = torch.zeros((p.rows, p.cols), dtype=torch.bfloat16, device=DEV)
    mxq.moe_expert_matmul_mxfp4(**d, residual=res, out=plain, expected_m=hint)
    d["q"], _ = wide(d["q"], 16, 32)
    d["scales"], _ = wide(d["scales"], 3, 2)
    ws = torch.full((3, 272, 8 + 16), 255, dtype=torch.uint8, device=DEV)
    ws[:, :, 8:19] = d["w_scales"]
    d["w_scales"] = ws[:, :, 8:19]
    res, _ = wide(res, 8, 8)
    out, big = wide(torch.zeros_like(plain), 8, 16)
    mxq.moe_expert_matmul_mxfp4(**d, residual=res, out=out, expected_m=hint)
    assert torch.equal(out, plain)
    assert (big[:, :8] == 0x7F).all() and (big[:, 8 + p.cols:] == 0x7F).all()
    # in place over the residual
    mxq.moe_expert_matmul_mxfp4(**d, residual=res, out=res, expected_m=hint)
    live = torch.from_numpy(p.live).to(DEV)
    assert torch.equal(res[live], plain[live])
    # quantized output into wider rows
    p = Problem(31, [20, 3, 150], 256, 384, fmt)
    d = p.dev()
    live = torch.from_numpy(p.live).to(DEV)
    for out_fmt, pay in (("mxfp4", 128), ("e8m0_g32", 256)):
        a, b = mxq.moe_expert_matmul_mxfp4_quant(
            **{**d, "act": "none"}, out_fmt=out_fmt, expected_m=hint)
        qo, qb = wide(torch.zeros((p.rows, pay), dtype=torch.uint8,
                                  device=DEV), 16, 32, 0xA5)
        so, sb = wide(torch.zeros((p.rows, 8), dtype=torch.uint8,
                                  device=DEV), 1, 2, 0xA5)
        mxq.moe_expert_matmul_mxfp4_quant(
            **{**d, "act": "none"}, out_fmt=out_fmt, q_out=qo, scales_out=so,
            expected_m=hint)
        assert torch.equal(qo[live], a[live]) and \
            torch.equal(so[live], b[live])
        assert (qb[:, :16] == 0xA5).all() and \
            (qb[:, 16 + pay:] == 0xA5).all()
        assert (sb[:, 0] == 0xA5).all() and (sb[:, 9:] == 0xA5).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act,N", [("none", 132), ("none", 4),
                                   ("silu_mul", 1432), ("silu_mul", 264)])
def test_rows_on_8_bytes(act, N, fmt):
    p = Problem(59, [20, 3, 140], N, 352, fmt, act, bias=True, residual=True,
                exact=act == "none")
    check_bf16(p, exact=act == "none")
    d = p.dev()
    out = torch.full((p.rows, p.cols + 8), 5.0, dtype=torch.bfloat16,
                     device=DEV)
    live = torch.from_numpy(p.live).to(DEV)
    for hint in HINTS:
        plain = mxq.moe_expert_matmul_mxfp4(**d, expected_m=hint)
        mxq.moe_expert_matmul_mxfp4(**d, out=out[:, 4:4 + p.cols],
                                    expected_m=hint)
        assert torch.equal(out[:, 4:4 + p.cols][live], plain[live])
        assert (out[:, :4] == 5).all() and (out[:, 4 + p.cols:] == 5).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_shapes_at_the_ends(fmt):
    p = Problem(41, [0, 0], 64, 128, fmt, pad=0)
    d = p.dev()
    out = torch.full((p.rows, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    mxq.moe_expert_matmul_mxfp4(**d, out=out)
    assert (out == 5).all()
    d["q"], d["scales"] = d["q"][:0], d["scales"][:0]
    assert mxq.moe_expert_matmul_mxfp4(**d).shape == (0, 64)
    check_bf16(Problem(43, [1], 8, 32, fmt, exact=True), exact=True)
    check_bf16(Problem(44, [3], 4, 32, fmt, exact=True), exact=True)
    counts = [(i * 7) % 4 for i in range(1024)]
    check_bf16(Problem(47, counts, 8, 32, fmt, pad=1, exact=True),
               HINTS + MANY_HINTS, exact=True)
    # the widest rows
    for H in (20320, 32768):
        check_bf16(Problem(48, [3, 40], 64, H, fmt, exact=True), exact=True)
    check_bf16(Problem(49, [3, 40] * 65, 12, 32768, fmt, pad=0, exact=True),
               MANY_HINTS, exact=True)


def test_as_quantized():
    """Weights and rows as the quantizer leaves them, one weight row per
    expert, and the fp8 product on widened rows."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((50, 352), generator=g).bfloat16().to(DEV)
    w = torch.randn((3, 64, 352), generator=g).to(DEV)
    q, s = mxq.mxfp4_quant_rows(x)
    wq, ws = mxq.mxfp4_quant_rows(w)
    off, n = i32_to_dev([0, 20, 21, 50]), i32_to_dev([20, 1, 29])
    y = mxq.moe_expert_matmul_mxfp4(q, s, wq, ws, off, n)
    want, err = mx.expert_matmul(host(q), host(s), "mxfp4", host(wq),
                                 host(ws), host(off), host(n), None, "none",
                                 None, 64)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + err) +
            err).all()
    q8 = mxq.mxfp4_to_e4m3(q)
    y8 = mxq.moe_expert_matmul_mxfp4(q8, s, wq, ws, off, n, fmt="e8m0_g32")
    got = y8.double().cpu().numpy()
    want, err = mx.expert_matmul(host(q8), host(s), "e8m0_g32", host(wq),
                                 host(ws), host(off), host(n), None, "none",
                                 None, 64)
    assert (np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + err) +
            err).all()
    # four columns of weights
    ws4 = torch.zeros((3, 4, 16), dtype=torch.uint8, device=DEV)[:, :, :11]
    ws4.copy_(ws[:, :4])
    y4 = mxq.moe_expert_matmul_mxfp4(q, s, wq[:, :4].contiguous(), ws4, off,
                                     n)
    assert torch.equal(y4, y[:, :4])


def test_refusals():
    p = Problem(53, [4, 6], 128, 352, "mxfp4")
    d = p.dev()

    def call(quant=False, **kw):
        a = {**d, **kw}
        if quant:
            return mxq.moe_expert_matmul_mxfp4_quant(**a)
        return mxq.moe_expert_matmul_mxfp4(**a)

    call()
    for kw in (dict(w=d["w"][:, :, :128].contiguous()),
               dict(w=d["w"][:, :, :80]),
               dict(w_scales=d["w_scales"].contiguous()),   # rows of 11 bytes
               dict(w_scales=d["w_scales"][:, :, :8]),
               dict(w_scales=d["w_scales"].contiguous()[:, :, :11]),
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
               dict(w=d["w"].cpu()), dict(fmt="e8m0_g32")):
        with pytest.raises(ValueError):
            call(**kw)
    # the last row's four bytes are not all there
    flat = torch.zeros(2 * 128 * 12 - 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        call(w_scales=flat.as_strided((2, 128, 11), (128 * 12, 12, 1)))
    for kw in (dict(q=d["q"].float()), dict(scales=d["scales"].int()),
               dict(out=torch.zeros((p.rows, 128), device=DEV))):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(act="relu"), dict(fmt="ue8m0_g128")):
        with pytest.raises(KeyError):
            call(**kw)
    with pytest.raises(KeyError):
        call(quant=True, out_fmt="ue8m0_g128")
    with pytest.raises(mxq.MxqError):
        call(expected_m=-1)
    with pytest.raises(mxq.MxqError):   # 64 + 16 gated columns
        call(quant=True, act="silu_mul", w=torch.zeros(
            (2, 160, 176), device=DEV, dtype=torch.uint8),
            w_scales=torch.zeros((2, 160, 12), device=DEV,
                                 dtype=torch.uint8)[:, :, :11])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hint", (1, 1 << 20))
def test_rows_far_apart(hint, fmt):
    """Rows, scales, residual and output beyond 2^32 bytes of their starts:
    the widest row strides the call takes."""
    p = Problem(61, [20, 300], 128, 256, fmt, residual=True, exact=True)
    d = p.dev()
    res = p.res.to(DEV)
    plain = mxq.moe_expert_matmul_mxfp4(**d, residual=res, expected_m=hint)
    rows, ld, at = 1400, 1 << 22, 1060  # expert 1 begins past 2^32 bytes
    a, b = int(p.offsets[1]), int(p.counts[1])
    src = torch.cat([torch.arange(20), torch.arange(a, a + b)]).to(DEV)
    dst = torch.cat([torch.arange(20), torch.arange(at, at + b)]).to(DEV)

    def far(t):
        big = torch.empty((rows, ld // t.element_size()), dtype=t.dtype,
                          device=DEV)[:, :t.shape[1]]
        big[dst] = t[src]
        return big

    say("mxfp4 rows far apart", hint, fmt)
    d["q"], d["scales"], res = far(d["q"]), far(d["scales"]), far(res)
    d["expert_offsets"] = i32_to_dev([0, at, at + b])
    out = far(torch.zeros_like(plain))
    mxq.moe_expert_matmul_mxfp4(**d, residual=res, out=out, expected_m=hint)
    assert torch.equal(out[dst], plain[src])
