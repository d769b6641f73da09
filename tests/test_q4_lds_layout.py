"""Shared memory of the 4-bit decode kernel: every part begins at a multiple of the
widest access made to it (16 bytes for the image and the kept sums), behind the part
before, for every batch, run of column tiles and workgroup.  The header that the
kernel and its plan use is compiled for the host."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "binary_rank_gemv_packed_amd", "csrc")
SOURCE = """
#include "nq_q4_lds.h"
extern "C" void layout(int P, int B, int tiles, int W, int keep, size_t* out) {
  const nq::Q4DecLds l = nq::q4_dec_lds(P, B, tiles, W, keep);
  out[0] = l.fac, out[1] = l.red, out[2] = l.total;
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("q4_lds")
    (d / "layout.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "layout.cpp"), "-o", str(d / "l.so")],
                   check=True)
    fn = ctypes.CDLL(str(d / "l.so")).layout
    out = (ctypes.c_size_t * 3)()

    def call(*args):
        fn(*args, out)
        return list(out)
    return call


@pytest.mark.parametrize("P", [1, 2])
@pytest.mark.parametrize("B", range(1, 17))
def test_parts_are_aligned_and_apart(layout, P, B):
    for tiles in (1, 2, 3, 5, 33, 64, 86, 224):
        for W in (1, 3, 4, 8, 16):
            for keep in (0, 1, 7):
                fac, red, total = layout(P, B, tiles, W, keep)
                assert red % 16 == 0 and fac % 4 == 0
                assert fac >= P * tiles * B * 128 * 2
                assert red - fac >= tiles * B * 4
                assert total - red >= keep * W * B * 16 * 4
