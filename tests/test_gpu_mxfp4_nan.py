"""e2m1 has no NaN: a group that holds one gets scale byte 255, which makes
all of it NaN again in what reads it."""
import numpy as np
import pytest
import torch

import fp8_mx_activation_amd as mxq
import mx_refs as mx
from gpu_util import DEV, assert_equal, host, i32_to_dev, say

pytestmark = pytest.mark.gpu
RULES = ("no_clip", "ocp_floor")


def rows_with_nans(dtype):
    """Rows, and [rows, groups]: which groups hold a NaN."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn((40, 96), generator=g)
    bits = [0x7FC00000, 0x7F810000, 0x7FFF0000, -0x400000, -0x10000]
    if dtype == torch.float32:
        bits += [0x7F800001, -0x7FFFFF]
    nan = torch.zeros((40, 3), dtype=torch.bool)
    at = torch.randperm(40 * 96, generator=g)[:30].tolist()
    xb = x.to(dtype).view(torch.int32 if dtype == torch.float32
                          else torch.int16)
    for i, k in enumerate(at):
        b = bits[i % len(bits)]
        xb[k // 96, k % 96] = b if dtype == torch.float32 else b >> 16
        nan[k // 96, k % 96 // 32] = True
    x = xb.view(dtype)
    assert torch.equal(torch.isnan(x).view(40, 3, 32).any(-1), nan)
    return x, nan


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows(dtype, rule):
    x, nan = rows_with_nans(dtype)
    say("mxfp4 NaN rows", dtype, rule)
    clean = torch.where(torch.isnan(x), torch.zeros_like(x), x)
    wq, ws = mx.quant(clean.double().numpy(), rule)
    gone = nan.numpy()

    def check(q, s):
        assert (host(s)[gone] == 255).all()
        assert_equal(host(s)[~gone], ws[~gone], "scales")
        keep = np.repeat(~gone, 16, 1)
        assert_equal(host(q)[keep], wq[keep], "payload")
        up = mxq.upscale_mxfp4_to_bf16(q, s).cpu()
        assert torch.equal(torch.isnan(up), nan.repeat_interleave(32, 1))

    check(*mxq.mxfp4_quant_rows(x.to(DEV), rule))
    if dtype == torch.bfloat16:
        s2d = torch.arange(40, dtype=torch.int32, device=DEV).view(-1, 1)
        check(*mxq.moe_scatter_quant_mxfp4(x.to(DEV), s2d, 40, rule))


@pytest.mark.parametrize("fmt", ["mxfp4", "e8m0_g32"])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("E", [2, 140])  # few blocks and many
def test_products(E, act, fmt):
    """Scale byte 255 of a row and of a weight row, through a quantized
    product and the next one."""
    g = torch.Generator().manual_seed(E)
    N, H, per = 256, 96, 20
    cols = N // 2 if act == "silu_mul" else N
    x = torch.randn((E * per, H), generator=g).bfloat16().to(DEV)
    q, s = mxq.mxfp4_quant_rows(x)
    if fmt != "mxfp4":
        q = mxq.mxfp4_to_e4m3(q)
    w, ws = mxq.mxfp4_quant_rows(torch.randn((E, N, H), generator=g).to(DEV))
    w2, ws2 = mxq.mxfp4_quant_rows(
        torch.randn((E, 64, cols), generator=g).to(DEV))
    row, weight = per + 3, 77
    s[row, 1] = 255
    ws[1, weight, 2] = 255
    off = i32_to_dev([i * per for i in range(E + 1)])
    cnt = i32_to_dev([per] * E)
    want = torch.zeros((E * per, cols // 32), dtype=torch.bool)
    want[row] = True
    want[per:2 * per, weight // 32] = True
    for hint in (1, 7, 13, 18, 40, 1 << 20):
        say("mxfp4 NaN products", E, act, fmt, hint)
        qo, so = mxq.moe_expert_matmul_mxfp4_quant(
            q, s, w, ws, off, cnt, fmt=fmt, act=act, expected_m=hint)
        assert torch.equal((so == 255).cpu(), want), hint
        y = mxq.moe_expert_matmul_mxfp4(qo, so, w2, ws2, off, cnt,
                                        expected_m=hint).cpu()
        assert torch.equal(torch.isnan(y).all(1), want.any(1))
        assert torch.equal(torch.isnan(y).any(1), want.any(1))
