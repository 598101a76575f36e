"""Tiles of an expert's rows, up to the most rows that a product takes.  The
compiler evaluates the kernels' own function: an overflow is an error there."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_mx_activation_amd", "csrc")
MOST = (1 << 31) - (1 << 16)  # MXQ_MAX_MATMUL_ROWS
COUNTS = (0, 1, 127, 128, 129, 256, 257, (1 << 30) - 1, 1 << 30,
          (1 << 30) + 1, 3 << 29, MOST - 1, MOST)


def compiles(lines):
    src = '#include "row_tiles.hpp"\n' + "\n".join(lines)
    gxx = shutil.which("g++") or pytest.skip("no host compiler")
    r = subprocess.run([gxx, "-std=c++17", "-I", CSRC, "-x", "c++",
                        "-fsyntax-only", "-"], input=src, text=True,
                       stderr=subprocess.PIPE)
    return r.returncode == 0, r.stderr


@pytest.mark.parametrize("tm", [128, 256, 0])
def test_row_tiles(tm):
    """Tiles of 128 and 256 rows; 0: one tile of all rows."""
    want = [-(-c // tm) if tm else int(c > 0) for c in COUNTS]
    ok, err = compiles('static_assert(mxq::row_tiles<%d>(%d) == %d, "");'
                       % (tm, c, n) for c, n in zip(COUNTS, want))
    assert ok, err


def test_no_tile_size_overflows():
    ok, _ = compiles(["constexpr int n = mxq::row_tiles<1 << 30>(1);"])
    assert not ok


def test_kernels_count_by_it():
    """No other rounding up of row counts in the products' kernels."""
    for name in ("matmul_device.hpp", "matmul.hip", "matmul_mxfp4.hip"):
        src = open(os.path.join(CSRC, name)).read()
        assert "+ TM - 1" not in src, name
