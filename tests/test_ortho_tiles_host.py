"""The lists of test_ortho_tiles_gpu.py reach every kernel that the choice of tiles has (CPU only)."""
from test_ortho_path_host import plan, program  # noqa: F401
from test_ortho_tiles_gpu import JOINED, LISTS, turned

KINDS = {"64", "128", "128 two", "192", "256"}
NAMES = ["64", "128", "128 two", "192", "256"]


def chosen(program, shapes):
    """(tile of A, of the squares, of X, joined) of a list, in the order in which the products take it."""
    by_n, _ = plan(program, *sorted(shapes, key=lambda s: -max(s)))
    by_m, sizes = plan(program, *sorted(shapes, key=lambda s: -min(s)))
    assert not all(s[4] for s in sizes)               # one workgroup would take them whole
    return NAMES[by_n[0]], NAMES[by_m[1]], NAMES[by_m[2]], bool(by_m[3])


def test_every_tile_is_reached(program):  # noqa: F811
    found = [chosen(program, s) for s in LISTS]
    assert [chosen(program, turned(s)) for s in LISTS] == found
    assert {f[0] for f in found} == {f[1] for f in found} == {f[2] for f in found} == KINDS
    # and the square with two addends, of the joined first steps
    assert {f[1] for f in found if f[3]} == KINDS
    assert ("256", "192", "256", True) in found       # as a large block's weights


def test_the_list_of_the_joined_steps(program):  # noqa: F811
    assert chosen(program, [JOINED])[3] and chosen(program, [(7700, 1920)])[3]
    assert not any(chosen(program, [s])[3] for s in ((85, 2715), (209, 309)))
