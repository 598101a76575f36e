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
