"""How far the products on 4-bit weights are from exact ones on rows as a layer
has them (normal values, quantized), for every kernel; and scales at the ends of
their range.

Of e4m3 rows the matrix unit drops what lies more than 13 bits below the largest
of the 32 products that it aligns, so each product is off by less than u = 2^-13
of that, which is at most 2^-13 of the largest of the 128 products of any step
that holds them.  Signs are random: a sum's variance is at most 32 u^2 over its
groups of 32, and E, its root, bounds the standard deviation; 8 E is what any of
10^5 outputs is off.  Products of e2m1 with e2m1 lose nothing there.  fp32's own
steps: H / 64 additions or fewer, half of 2^-23 of a partial sum each, which
hardly passes the result's size or the outputs' root mean square: at most their
number times 2^-24 of both together."""
import pytest
import torch

import fp8_mx_activation_amd as mxq
import mx_refs as mx
from gpu_util import DEV, host, i32_to_dev, say

pytestmark = pytest.mark.gpu

H = 7168
# rows of every expert, weight rows, hints that reach each kernel: the K split
# and both tiles for few blocks; the stream of 128 and of 256 weight rows and
# the tiles for many
FEW = ([150], 384, (1, 40, 1 << 20))
MANY = ([3, 1, 0, 17] * 33, 256, (1, 7, 13, 18, 1 << 20))


def problem(counts, N, fmt, seed):
    """Device inputs and the exact sums with E, in 64 bits, row by row."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    E, R = len(counts), sum(counts)
    x = torch.randn((R, H), generator=gen, device=DEV).bfloat16()
    s2d = torch.arange(R, dtype=torch.int32, device=DEV).view(-1, 1)
    if fmt == "mxfp4":
        q, s = mxq.moe_scatter_quant_mxfp4(x, s2d, R)
    else:
        q, s = mxq.moe_scatter_quant(x, s2d, R, fmt=fmt)
        s = s.view(torch.uint8)
    w = torch.randn((E, N, H), generator=gen, device=DEV) / H ** 0.5
    w, ws = mxq.mxfp4_quant_rows(w)
    xd = torch.from_numpy(mx.values(host(q.view(torch.uint8)), host(s),
                                    fmt)).to(DEV)
    table = torch.from_numpy(mx.E2M1).to(DEV)
    offsets = [0]
    a = torch.zeros((R, N), dtype=torch.float64, device=DEV)
    var = torch.zeros_like(a)
    for e, n in enumerate(counts):
        offsets.append(offsets[-1] + n)
        if not n:
            continue
        b = w[e].int()
        wd = table[torch.stack([b & 15, b >> 4], -1).reshape(N, H)] * \
            torch.exp2(ws[e].double() - 127).repeat_interleave(32, 1)
        at = slice(offsets[e], offsets[e + 1])
        a[at] = xd[at] @ wd.t().contiguous()
        if fmt != "mxfp4":
            xa, wa = xd[at].abs(), wd.abs()
            for k in range(0, H, 128):
                u = torch.zeros_like(a[at])
                for c in range(k, k + 128):
                    torch.maximum(u, xa[:, c, None] * wa[None, :, c], out=u)
                var[at] += 4 * 32 * (2.0 ** -13 * u) ** 2
    rms = a.pow(2).mean().sqrt()
    err = var.sqrt() + H / 64 * 2.0 ** -24 * (a.abs() + rms)
    d = dict(q=q, scales=s, w=w, w_scales=ws,
             expert_offsets=i32_to_dev(offsets), counts=i32_to_dev(counts),
             fmt=fmt)
    return d, a, err


@pytest.mark.parametrize("fmt", ["mxfp4", "e8m0_g32"])
@pytest.mark.parametrize("which", ["few", "many"])
def test_error_of_normal_rows(which, fmt):
    counts, N, hints = FEW if which == "few" else MANY
    d, a, E = problem(counts, N, fmt, len(counts))
    for hint in hints:
        # what bf16 leaves of the result is taken off in the epilogue (the
        # difference is exact in fp32), so its rounding is that of the rest
        near = a.to(torch.bfloat16)
        out = mxq.moe_expert_matmul_mxfp4(**d, residual=-near,
                                          expected_m=hint).double()
        off = out - (a - near.double())
        step = 2.0 ** -8 * out.abs()
        rel = (off.norm() / a.norm()).item()
        say("error of normal rows", which, fmt, hint, "%.2e" % rel,
            "bound %.2e" % (E.norm() / a.norm()).item())
        assert (off.abs() <= 8 * E + step).all()
        assert off.norm() <= E.norm() + step.norm()
        # measured 5.0e-6 of 8-bit rows and 0 of 4-bit ones (whose sums fp32
        # holds) for every kernel; equal calls give equal bytes
        assert rel <= 1e-5


@pytest.mark.parametrize("fmt", ["mxfp4", "e8m0_g32"])
@pytest.mark.parametrize("which", ["few", "many"])
def test_scales_that_cancel(which, fmt):
    """Rows times 2^k with weights times 2^-k: the same bytes, up to where the
    scale bytes end, for every kernel."""
    counts, N, hints = FEW if which == "few" else MANY
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    R, E, h = sum(counts), len(counts), 352
    q, s = mxq.mxfp4_quant_rows(torch.randn((R, h), generator=gen,
                                            device=DEV))
    if fmt != "mxfp4":
        q = mxq.mxfp4_to_e4m3(q)
    w, ws = mxq.mxfp4_quant_rows(torch.randn((E, N, h), generator=gen,
                                             device=DEV))
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    off, cnt = i32_to_dev(off), i32_to_dev(counts)
    top = 254 - max(int(s.max()), int(ws.max()))
    low = min(int(s.min()), int(ws.min())) - 1
    for hint in hints:
        say("scales that cancel", which, fmt, hint)
        want = mxq.moe_expert_matmul_mxfp4(q, s, w, ws, off, cnt, fmt=fmt,
                                           expected_m=hint)
        for k in (1, 60, min(top, low), -min(top, low)):
            big = torch.full((E, N, 16), 127, dtype=torch.uint8, device=DEV)
            ws2 = big[:, :, :h // 32]
            ws2.copy_(ws.int() - k)
            got = mxq.moe_expert_matmul_mxfp4(
                q, (s.int() + k).to(torch.uint8), w, ws2, off, cnt, fmt=fmt,
                expected_m=hint)
            assert torch.equal(got, want), (hint, k)
