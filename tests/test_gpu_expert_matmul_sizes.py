"""The experts' products where the kernels' bookkeeping begins: rows of
channels that take several chunks of scales (and use a chunk's place again),
the few-row kernel with 256 weight rows to a block over several steps, and more
row tiles than share a column of weights.  Bit for bit where every sum is
exact in fp32 (payloads of two exponents and scales of three: sums of up to
32768 random signs stay below 2^16, in steps of 2^-8)."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_expert_matmul import Problem, check_bf16, check_quant


pytestmark = pytest.mark.gpu

G128, G32 = "ue8m0_g128", "e8m0_g32"


@pytest.mark.parametrize("fmt,H", [(G128, 4096), (G128, 4224), (G128, 8320),
                                   (G32, 1024), (G32, 2080), (G32, 3136),
                                   (G128, 32768), (G32, 32768)])
def test_many_scale_chunks(fmt, H):
    counts = [5, 0, 140, 20]
    say("scale chunks", fmt, H)
    check_bf16(Problem(H, counts, 136, H, fmt, bias=True, residual=True,
                       exact=True), exact=True)
    if H > 8320:
        return
    check_bf16(Problem(H + 1, counts, 272, H, fmt, "silu_mul", bias=True))
    check_quant(Problem(H + 2, counts, 256, H, fmt, "silu_mul"), G128)
    check_quant(Problem(H + 3, counts, 96, H, fmt, "silu"), G32)


# experts enough for 256 weight rows to a block, one with more rows than the
# few-row kernel takes at a time
WIDE = [(i * 5) % 4 for i in range(60)] + [0, 40, 1, 17]


@pytest.mark.parametrize("fmt,H", [(G128, 640), (G32, 672)])
@pytest.mark.parametrize("N", [1032, 1280])
def test_few_rows_of_wide_experts(N, fmt, H):
    assert -(-N // 256) * len(WIDE) >= 256
    say("wide experts", N, fmt, H)
    check_bf16(Problem(N, WIDE, N, H, fmt, bias=True, residual=True,
                       exact=True), hints=(1, 12, 13), exact=True)
    check_bf16(Problem(N + 1, WIDE, N, H, fmt, "silu", bias=True),
               hints=(1,))


@pytest.mark.parametrize("fmt,H", [(G128, 640), (G32, 672)])
def test_few_rows_of_wide_gated_experts(fmt, H):
    say("wide gated experts", fmt, H)
    check_bf16(Problem(3, WIDE, 1040, H, fmt, "silu_mul", bias=True,
                       residual=True), hints=(1, 12))


@pytest.mark.parametrize("fmt,H", [(G128, 640), (G32, 672)])
@pytest.mark.parametrize("act,out_fmt,cols", [
    ("none", G32, 1056), ("none", G128, 1152), ("silu_mul", G32, 544),
    ("silu_mul", G128, 1152)])
def test_few_rows_of_wide_experts_quantized(act, out_fmt, cols, fmt, H):
    N = cols * 2 if act == "silu_mul" else cols
    assert -(-N // 256) * len(WIDE) >= 256
    say("wide experts, quantized", act, out_fmt, cols, fmt, H)
    check_quant(Problem(cols, WIDE, N, H, fmt, act, bias=True), out_fmt,
                hints=(1, 12))


@pytest.mark.parametrize("fmt", [G128, G32])
@pytest.mark.parametrize("counts", [
    [1034, 0, 700, 900, 1, 300],             # 15 row tiles of 256, 27 of 128
    [2048, 2048],                            # whole groups of eight, 16 and 32
    [200] * 11,                              # 11 and 22
    [0, 2300, 0]])                           # 9 and 18 of one expert
def test_groups_of_row_tiles(counts, fmt):
    """Three columns of tiles over one to four groups of row tiles."""
    say("groups of row tiles", counts, fmt)
    check_bf16(Problem(len(counts), counts, 600, 256, fmt, bias=True,
                       residual=True, exact=True), hints=(13, 1 << 20),
               exact=True)
    check_bf16(Problem(len(counts), counts, 720, 256, fmt, "silu_mul"),
               hints=(13, 1 << 20))


def test_row_tiles_of_many_experts():
    """More experts than a wavefront's lanes, several tiles each: 150 row
    tiles of 128 and 125 of 256, three columns."""
    counts = [(i * 37) % 300 for i in range(100)]
    say("row tiles of many experts")
    p = Problem(9, counts, 520, 128, G128, exact=True, pad=2)
    assert np.sum(-(-p.counts // 256)) > 100
    check_bf16(p, hints=(13, 1 << 20), exact=True)
