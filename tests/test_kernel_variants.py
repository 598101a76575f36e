"""Variants of the kernels that no call reaches are not compiled."""
import os

import fp8_mx_activation_amd as mxq


def test_ring_of_4_bit_rows():
    """The K split on 4-bit rows always holds three steps: its kernels are
    <false, 3, OUT>, never <false, 2, OUT>."""
    if not os.path.exists(mxq.LIB_PATH):
        from fp8_mx_activation_amd import build
        build.build(verbose=False)
    lib = open(mxq.LIB_PATH, "rb").read()
    name = b"matmul4_small_kernelILb%dELi%dE"
    for x8, ring, there in ((1, 2, True), (1, 3, True), (0, 3, True),
                            (0, 2, False)):
        assert (name % (x8, ring) in lib) == there, (x8, ring)
