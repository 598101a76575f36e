"""Calls that need more threads than one launch holds (2^32 - 1) are refused
before anything is enqueued; the runtime would wrap them without an error."""
import os

import pytest

UNSUPPORTED = 2
FAKE = 1 << 20  # 16-byte aligned, never dereferenced by a refused call


@pytest.fixture(scope="module")
def lib():
    import fp8_mx_activation_amd as m
    if not os.path.exists(m.LIB_PATH):
        from fp8_mx_activation_amd import build
        build.build(verbose=False)
    return m.lib()


@pytest.mark.parametrize("rows,E,N,m", [
    ((1 << 31) - (1 << 16), 1024, 4, 13),    # row tiles of 128
    ((1 << 31) - (1 << 16), 1024, 1024, 1 << 30),
    (8, 1024, 1 << 25, 1)])                  # blocks of 256 weight rows
def test_expert_matmul(lib, rows, E, N, m):
    assert lib.moe_expert_matmul(
        FAKE, 32, FAKE, 1, rows, 1, FAKE, FAKE, E, N, 32, FAKE, FAKE, None, 0,
        None, 0, m, FAKE, N, None) == UNSUPPORTED


# calls whose blocks have 64 to 1024 threads, one to a row; the last one that
# fits is not made here, for it would go on to the launch
def test_row_kernels(lib):
    for H, T in ((128, 1 << 26), (8192, 1 << 22), (2048, 1 << 24)):
        assert lib.moe_combine(FAKE, H, 8, FAKE, FAKE, T, 1, H, FAKE, H, 0,
                               None) == UNSUPPORTED
    assert lib.moe_scatter_quant(FAKE, 128, 1 << 22, 128, FAKE, 1, 0, FAKE,
                                 128, FAKE, 1, 8, None) == UNSUPPORTED
    assert lib.moe_scatter_quant_mfma(
        FAKE, 128, (1 << 22) - 7, 128, FAKE, 1, 0, 0, FAKE, 128, FAKE, 32, 8,
        None) == UNSUPPORTED
    assert lib.moe_scatter_rows(
        FAKE, 128, 1 << 23, 128, None, 0, 0, 0, 1, FAKE, 1, 8, FAKE, 128,
        None, 0, 0, None) == UNSUPPORTED
    assert lib.upscale_fp8_to_bf16(FAKE, 128, FAKE, 1, 1, 1 << 26, 128, 128,
                                   FAKE, 128, None) == UNSUPPORTED
    assert lib.mxq_gather_read16(FAKE, 16, 8, FAKE, 1 << 26, 1, 16, FAKE,
                                 None) == UNSUPPORTED
    assert lib.mxq_fill_rows16(FAKE, 16, 1 << 26, 16, 0, None) == UNSUPPORTED


def test_weight_requant(lib):
    n = 1 << 23  # blocks of 512 threads, one to a matrix of one block
    assert lib.requant_weight_block_ue8m0(
        FAKE, 16, 16, FAKE, 1, 1, n, 1, 16, 128, 128, FAKE, FAKE, 1, 1,
        None) == UNSUPPORTED


def test_live_rows_segments(lib):
    """Above 1024 segments each has a block of its own."""
    n, H = 1 << 22, 16384
    assert lib.mx_quant_live_rows(FAKE, H, n, 1, FAKE, H, 1, FAKE, H, FAKE,
                                  H // 32, None) == UNSUPPORTED
