"""Which kernel an 8-bit product takes (CPU only): the choice is plain host C++ (csrc/fp8_path.h), compiled here with g++."""
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_fp4_hadamard_amd", "csrc")
PATHS = ["few", "mid", "big"]

SRC = r"""
#include "fp8_path.h"
#include <cstdio>
#include <cstdlib>
int main(int argc, char** argv) {
  // args: M N K lda ldb tile_scales exact, repeated; out: path, splits, rounds, columns of the kernel for few rows
  for (int a = 1; a + 6 < argc; a += 7) {
    long long v[7];
    for (int i = 0; i < 7; ++i) v[i] = strtoll(argv[a + i], 0, 0);
    const mx::Fp8Plan p = mx::fp8_plan(v[0], v[1], v[2], v[3], v[4], v[5], v[6] != 0);
    printf("%d %d %d %d\n", (int)p.path, p.splits, p.path == mx::Fp8Path::kBig ? p.big.rounds : 0,
           mx::fp8_few_columns(v[0], v[1], v[6] != 0));
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plans():
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tempfile.mkdtemp()
    src, exe = os.path.join(d, "p.cpp"), os.path.join(d, "p")
    with open(src, "w") as f:
        f.write(SRC)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I" + CSRC, src, "-o", exe])

    def run(cases):
        args = [exe] + [str(int(x)) for c in cases for x in c]
        rows = [[int(t) for t in line.split()] for line in subprocess.check_output(args).decode().splitlines()]
        return [(PATHS[path], splits, rounds, columns) for path, splits, rounds, columns in rows]
    yield run
    shutil.rmtree(d, ignore_errors=True)


def case(M, N, K, lda=None, ldb=None, tile_scales=0, exact=False):
    k = -(-K // 128) * 128
    return (M, N, K, k if lda is None else lda, k if ldb is None else ldb, tile_scales, exact)


def test_pitches_that_the_tiled_kernels_cannot_address_take_the_kernel_for_few_rows(plans):
    far = 1 << 24
    got = plans([case(300, 500, 1000), case(300, 500, 1000, lda=far - 16, ldb=far - 16), case(300, 500, 1000, lda=far),
                 case(300, 500, 1000, ldb=far), case(300, 500, far - 128), case(300, 500, far + 1),
                 case(300, 500, 1000, tile_scales=(1 << 30) - 1), case(300, 500, 1000, tile_scales=1 << 30)])
    assert [g[0] for g in got] == ["mid", "mid", "few", "few", "mid", "few", "mid", "few"]


def test_many_lines_take_a_tiled_kernel(plans):
    """Line scales are at least as far apart as there are lines; that says nothing about the codes' rows.  2^24 rows, 32
    at a time, would be 524288 launches."""
    shapes = [((1 << 24) + 77, 24, 128), (24 * 32, (1 << 24) + 5, 128), (1 << 26, 8, 256)]
    assert all(g[0] != "few" for exact in (False, True) for g in plans([case(*s, exact=exact) for s in shapes]))


def test_shapes_of_the_gpu_tests_take_the_kernels_they_are_meant_for(plans):
    from test_fp8_large_gpu import BIG, FAR, FAR_SHAPES, SMALL_SCALES, chunks
    for (m, n, k), which, path in FAR_SHAPES:
        packed, far = plans([case(m, n, k), case(m, n, k, lda=FAR if which in ("a", "both") else None,
                                                 ldb=FAR if which in ("b", "both") else None, tile_scales=1 << 20)])
        assert packed[0] == far[0] == path, (m, n, k)
    assert [g[0] for g in plans([case(*s) for s in SMALL_SCALES])] == ["few", "few", "mid", "mid", "big"]
    assert plans([case(*SMALL_SCALES[3])])[0][1] > 1
    large = plans([case(*s) for s in BIG + [(4096, 8192, 4096)]])
    assert all(g[0] == "big" for g in large) and min(g[2] for g in large) == 1 and max(g[2] for g in large) >= 4
    for m, n, k in BIG:
        parts = chunks(m, n)
        covered = np.zeros(n, bool)
        for at, width in parts:
            covered[at:at + width] = True
        assert covered.all() and all(g[:2] == ("mid", 1) for g in plans([case(m, w, k) for _, w in parts]))


def test_the_grid_of_the_kernel_for_few_rows_fits_a_launch(plans):
    """512 threads for each 16 columns and fragment, fewer than 2^32 in all, up to the widest product the ABI takes."""
    cases = [case(M, N, 128, exact=exact) for M in (1, 2, 16, 17, 31, 32) for exact in (False, True)
             for N in (1, 16, 17, 4096, 128256, (1 << 26) + 1, (1 << 27) - 17, (1 << 27) - 1)]
    for c, (path, _, _, columns) in zip(cases, plans(cases)):
        assert path == "few" and 1 <= columns <= 4 and -(-c[1] // (16 * columns)) * 512 < 1 << 32, c
