"""Which bytes the 4-bit product's warps copy, on the host (no GPU): the library's own functions, compiled with g++.

Every 16-byte piece of every tile of 128 columns, those past the last column among them (a block has 256), has to lie
inside its row but for the bytes before the row in its first 16, and the pieces have to cover the row.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

from scatter_boundary_tile_gb300 import _build

SOURCE = r"""
#include "matvec_copies.h"
// Columns n0 .. n0 + 127 of a row of `row` bytes (`per` columns each) at address `at`, in pieces of 16 bytes.
// 0, or what is wrong: 1 a byte outside, 2 a byte that is missing, 3 a piece where there is no byte.
extern "C" int check(int64_t at, int64_t row, int64_t n0, int per, int tile) {
    const int bytes = sbt_matvec::bytes_of(row, n0 / per, tile);
    const int64_t src = at + n0 / per;
    const int shift = (int)(src & 15);
    int64_t covered = src;
    for (int c = 0; c < 512; c += 16) {
        const int n = sbt_matvec::piece_of(bytes, shift, c);
        const int64_t from = src - shift + c;
        if (n == 0) continue;
        if (bytes == 0) return 3;
        if (n > 16 || from + n > at + row || from < (src & ~int64_t(15))) return 1;
        if (from <= covered) covered = from + n;
    }
    const int64_t end = at + (n0 / per + tile < row ? n0 / per + tile : row);
    return src < end && covered < end ? 2 : 0;
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("copies")
    (d / "check.cc").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", _build.CSRC, str(d / "check.cc"), "-o",
                    str(d / "check.so")], check=True)
    f = ctypes.CDLL(os.path.join(d, "check.so")).check
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    return f


@pytest.mark.parametrize("per,tile", [(2, 64), (1, 128)])  # weights, two columns a byte; scales
def test_every_piece_of_every_tile(check, per, tile):
    for N in [*range(1, 300), 511, 512, 513, 1000, 1153]:
        row = -(-N // per)
        for at in range(4096, 4113):
            for n0 in range(0, -(-N // 256) * 256, 128):
                assert check(at, row, n0, per, tile) == 0, (N, at, n0)
