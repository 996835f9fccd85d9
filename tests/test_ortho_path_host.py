"""How a list of matrices is orthogonalized (CPU only): sizes, bounds and tiles are plain host C++ (csrc/ortho_path.h),
compiled here with g++."""
import os
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_fp4_hadamard_amd", "csrc")

SRC = r"""
#include "ortho_path.h"
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>
struct Item { long long rows, cols; };
int main(int argc, char** argv) {
  if (!strcmp(argv[1], "plan")) {            // rows cols, repeated: one list
    std::vector<Item> list;
    for (int a = 2; a + 1 < argc; a += 2) list.push_back({atoll(argv[a]), atoll(argv[a + 1])});
    std::vector<mx::OrthoSize> s;
    for (auto& t : list) s.push_back(mx::ortho_size(t.rows, t.cols));
    const int n = (int)s.size();
    printf("%d %d %d %d", (int)mx::ortho_choose(s.data(), n, true, true), (int)mx::ortho_choose(s.data(), n, true, false),
           (int)mx::ortho_choose(s.data(), n, false, false), (int)mx::ortho_joins(list.data(), n));
    for (auto& z : s) printf(" %lld %lld %lld %lld %d %lld", (long long)z.m, (long long)z.n, (long long)z.parts,
                             (long long)z.bytes, (int)mx::ortho_small_fits(z), (long long)mx::ortho_small_bytes(z));
    printf("\n");
  } else if (!strcmp(argv[1], "reach")) {    // a b c top
    const mx::OrthoReach r = mx::ortho_reach(atof(argv[2]), atof(argv[3]), atof(argv[4]), atof(argv[5]));
    printf("%.17g %.17g\n", r.x, r.factor);
  } else {                                   // groups: rows cols, repeated
    std::vector<Item> list;
    for (int a = 2; a + 1 < argc; a += 2) list.push_back({atoll(argv[a]), atoll(argv[a + 1])});
    mx::each_ortho_group(list.data(), (int)list.size(), [&](const int32_t* at, int n, int64_t bytes) {
      printf("%lld", (long long)bytes);
      for (int i = 0; i < n; ++i) printf(" %d", at[i]);
      printf("\n");
      return true;
    });
  }
  return 0;
}
"""
TILE = [64, 128, 128, 192, 256]


@pytest.fixture(scope="module")
def program():
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tempfile.mkdtemp()
    src, exe = os.path.join(d, "p.cpp"), os.path.join(d, "p")
    with open(src, "w") as f:
        f.write(SRC)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I" + CSRC, src, "-o", exe])
    return lambda *args: subprocess.check_output([exe] + [str(a) for a in args]).decode()


def plan(program, *shapes):
    v = [int(t) for t in program("plan", *[x for s in shapes for x in s]).split()]
    return v[:4], [v[4 + 6 * i:10 + 6 * i] for i in range(len(shapes))]


def test_every_tile_stays_inside_its_buffer(program):
    """Whole steps of 64, and room for what the last tile of any size passes them by; each part of the workspace at 16
    bytes."""
    for rows, cols in ((1, 1), (64, 64), (65, 1000), (1000, 65), (4096, 14336), (4097, 4095), (28672, 4096)):
        _, ((m, n, parts, size, _, _),) = plan(program, (rows, cols))
        assert (m, n) == tuple(sorted((-(-rows // 64) * 64, -(-cols // 64) * 64)))
        assert 1 <= parts <= 256
        for side in (m, n):
            for tile in (64, 128, 192, 256):
                assert -(-side // tile) * tile <= side + 192
        assert size == 8 * 256 + 2 * (3 * (m + 192) * (n + 192) + 3 * (m + 192) ** 2) and size % 16 == 0


def test_tiles_grow_with_the_work(program):
    """The tiles that were measured to be fastest: small ones spread little work over the chip, large ones reuse more."""
    def sides(*shapes):
        return [TILE[t] for t in plan(program, *shapes)[0][:3]]

    assert sides((512, 512)) == [64, 64, 64]
    assert sides((1024, 1024)) == [64, 64, 64]
    assert sides((2048, 2048)) == [128, 128, 128]
    assert sides((4096, 4096)) == [192, 192, 256]
    assert sides((4096, 14336)) == [192, 192, 256]
    assert sides((28672, 4096), (4096, 14336), (6144, 4096), (4096, 4096)) == [256, 192, 256]


def test_first_steps_join_where_matrices_are_wide(program):
    joins = lambda *s: plan(program, *s)[0][3]        # noqa: E731
    assert joins((4096, 14336)) and joins((28672, 4096)) and not joins((4096, 4096))
    assert joins((28672, 4096), (4096, 4096)) and not joins((128, 512))


def test_small_matrices_fit_one_workgroup(program):
    """Everything that passes the test fits into 160 KB of LDS, beside the workgroup's own 128 bytes."""
    for m in (64, 128):
        for n in range(m, 1089, 64):
            _, ((_, _, _, _, fits, size),) = plan(program, (m, n))
            assert fits == (m * n <= 32768)
            assert not fits or size + 128 <= 160 * 1024
    assert plan(program, (129, 64))[1][0][4] == 1 and plan(program, (129, 129))[1][0][4] == 0


def test_groups(program):
    out = [[int(t) for t in line.split()] for line in program("groups", *([100, 300] * 33 + [0, 5])).splitlines()]
    assert [g[1:] for g in out] == [list(range(32)), [32]]
    out = [[int(t) for t in line.split()] for line in
           program("groups", 28672, 4096, 0, 7, 4096, 14336, 28672, 4096, 5, 5).splitlines()]
    assert [g[1:] for g in out] == [[0, 2], [3, 4]]
    assert all(g[0] <= 1 << 31 for g in out)


def test_reach(program):
    """The closed form against a fine grid."""
    rng = np.random.default_rng(5)
    for a, b, c, top in [(3.4445, -4.7750, 2.0315, 1.0), (3.4445, -4.7750, 2.0315, 1.2), (1.5, -0.5, 0.0, 1.7),
                         (2.0, 0.0, 0.0, 1.0), (0.0, 0.0, 1.0, 2.0)] + [tuple(rng.uniform(-3, 3, 3)) + (1.5,)
                                                                        for _ in range(40)]:
        x, f = (float(t) for t in program("reach", a, b, c, top).split())
        s = np.linspace(0, top, 200001)
        t = s * s
        wx = np.abs(s * (a + b * t + c * t * t)).max()
        wf = max(np.abs(b * t + c * t * t).max(), np.abs(a + b * t + c * t * t).max())
        assert wx <= x * (1 + 1e-12) + 1e-300 and x <= wx * (1 + 1e-6) + 1e-12
        assert wf <= f * (1 + 1e-12) + 1e-300 and f <= wf * (1 + 1e-6) + 1e-12
