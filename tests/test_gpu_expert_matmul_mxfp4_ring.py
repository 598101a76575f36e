"""Rows of 8 bits on both sides of the length from which the K split holds two
steps of its ring instead of three: the scales of 16 rows have 10240 bytes of LDS,
in words and one more word each, 632 blocks of 32 channels."""
import pytest

from gpu_util import say
from test_gpu_expert_matmul_mxfp4 import Problem, check_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("H", [20192, 20224, 20256, 32768])
def test_ring(H, act):
    say("ring of 8-bit rows", H, act)
    check_bf16(Problem(H, [3, 17], 72, H, "e8m0_g32", act, bias=True,
                       exact=True), (1, 13, 24), exact=act == "none")
