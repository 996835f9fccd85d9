"""Every kernel of the Newton-Schulz products (tile, kind of product, side and epilogue) on the GPU against float64, place
by place; views, special values and the joined first steps through them.

test_ortho_tiles_host.py holds the lists here to the tiles that they are meant for.
"""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import MuonTensors, muon_step, orthogonalize
from gpu_helpers import announce
from oracle import ortho

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
OFF = 2.6e-3              # the documented error of such gradients, of the result's norm
A, B, C = ortho.COEFFICIENTS

# sizes that end inside tiles, vectors and K steps; between them every tile of every kind of product
LISTS = [
    [(333, 701), (701, 200)],
    [(206, 1484), (657, 487), (272, 781), (616, 345), (517, 798), (784, 391)],
    [(1356, 1987)],
    [(2039, 2506)],
    [(3712, 2374)],
    [(289, 1041), (2780, 3775)],
    [(2839, 3027)],
    [(1992, 1725), (2062, 2498), (1974, 1145)],
    [(3336, 3375), (5613, 2772)],
    [(3256, 2289), (428, 1847), (1656, 2557), (3180, 2519), (4307, 252), (2250, 1627)],
]
JOINED = (1070, 3460)     # its first two steps run as one


def turned(shapes):
    return [s[::-1] for s in shapes]


def gradient(rows, cols, seed, dtype):
    """A few strong directions over noise."""
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + rows + cols)
    left = torch.randn((rows, 24), generator=gen, device="cuda") / torch.arange(1, 25, device="cuda")
    g = left @ torch.randn((24, cols), generator=gen, device="cuda")
    return (1e-3 * (g + 0.1 * torch.randn((rows, cols), generator=gen, device="cuda"))).to(dtype)


def exact(u, steps=5, eps=1e-7):
    x = u.double()
    x = x / (torch.linalg.vector_norm(x) + eps)
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            s = x @ x.t().contiguous()
            x = A * x + (B * s + C * (s @ s)) @ x
        else:
            s = x.t().contiguous() @ x
            x = A * x + x @ (B * s + C * (s @ s))
    return x


def near(got, want, size, rate, own, what):
    """got off want by at most OFF of its norm, rate * `size` (plus `own`, elementwise: roundings of got itself), and no
    element by more than 16 times that: an element's error is a sum of many roundings, so of normal distribution, and its
    deviation in a row or column is less than three times the mean one.  A piece that is astray is off by its size, 1.4 /
    (16 OFF) = 33 times as much."""
    off = (got.double() - want).abs()
    rms = size / want.numel() ** 0.5
    assert float(torch.linalg.vector_norm(off)) <= rate * OFF * size + float(torch.linalg.vector_norm(own)), what
    assert bool((off <= 16 * OFF * rate * rms + own).all()), what


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("number", range(len(LISTS)))
def test_results_of_every_tile(number, turn):
    shapes = turned(LISTS[number]) if turn else LISTS[number]
    announce("ortho tiles %s" % shapes)
    gs = [gradient(*s, i, torch.bfloat16 if (i + number) % 2 else torch.float32) for i, s in enumerate(shapes)]
    dtype = torch.bfloat16 if turn == (number % 2 == 0) else torch.float32
    for g, got in zip(gs, orthogonalize(gs, out_dtype=dtype)):
        want = exact(g)
        near(got, want, float(torch.linalg.vector_norm(want)), 1.0, HALF[dtype] * 1.05 * want.abs() + 1e-6, tuple(g.shape))


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("number", range(len(LISTS)))
def test_muon_step_of_every_tile(number, turn):
    """Moments, weights and copies where the products' epilogue writes them, with a rate at which the update is the most
    of the new weight."""
    shapes = turned(LISTS[number]) if turn else LISTS[number]
    announce("muon tiles %s" % shapes)
    gen = torch.Generator(device="cuda").manual_seed(70 + number)
    gs = [gradient(*s, 30 + i, torch.float32 if (i + number) % 2 else torch.bfloat16) for i, s in enumerate(shapes)]
    ms = [gradient(*s, 60 + i, torch.float32) for i, s in enumerate(shapes)]
    ws = [0.02 * torch.randn(s, generator=gen, device="cuda") for s in shapes]
    hs = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") if i or turn else None for i, s in enumerate(shapes)]
    before = [[x.double() for x in t] for t in (ws, gs, ms)]
    muon_step(MuonTensors(ws, gs, ms, copies=hs), lr=1.0, momentum=0.9, weight_decay=0.2, adjust="plain")
    for w, g, m, h, w0, g0, m0 in zip(ws, gs, ms, hs, *before):
        m1 = 0.9 * m0 + 0.1 * g0
        # 0.9 and 0.1 as float32, two products, one sum
        assert bool(((m.double() - m1).abs() <= 4 * U * (0.9 * m0.abs() + 0.1 * g0.abs())).all()), tuple(g.shape)
        o = exact(0.1 * g0 + 0.9 * m1)
        near(w, 0.8 * w0 - o, float(torch.linalg.vector_norm(o)), 1.0, 3 * U * (w0.abs() + o.abs()) + 1e-6, tuple(g.shape))
        assert h is None or torch.equal(h, w.bfloat16())


@pytest.mark.parametrize("shape", [(300, 521), (521, 300), (1356, 1987), (2506, 2039)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_views_through_the_tiles(shape, dtype):
    """Pitches on both sides, and nothing written between the rows.  (The sum of squares is added in another order, in
    float64: the scale is the same float32.)"""
    announce("ortho tiles views %s %s" % (shape, dtype))
    rows, cols = shape
    g = gradient(rows, cols, 90, dtype)
    want = orthogonalize(g, out_dtype=dtype)
    buf = torch.full((rows + 10, cols + 31), 7.0, dtype=dtype, device="cuda")
    src = buf[3:3 + rows, 5:5 + cols]
    src.copy_(g)
    dst = torch.full((rows + 9, cols + 30), 5.0, dtype=dtype, device="cuda")
    out = dst[2:2 + rows, 7:7 + cols]
    assert orthogonalize(src, out=out) is out and torch.equal(out, want)
    out.fill_(5.0)
    assert bool((dst == 5.0).all())
    src.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("shape", [(300, 521), (1356, 1987), (2506, 2039)])
def test_special_values_through_the_tiles(shape):
    """NaN and Inf take their matrix and no other; the gradient's scale does not matter; eps does where it is as large as
    the norm."""
    announce("ortho tiles special %s" % (shape,))
    g = gradient(*shape, 91, torch.float32)
    for bad in (float("nan"), float("inf")):
        for at in ((shape[0] - 1, shape[1] - 1), (0, 0)):
            worse = g.clone()
            worse[at] = bad
            a, b = orthogonalize([worse, g])
            assert a.isnan().all() and b.isfinite().all()
    want = exact(g)
    size = float(torch.linalg.vector_norm(want))
    for scale in (2.0 ** 100, 2.0 ** -80):
        got = orthogonalize(g * scale, eps=1e-38, out_dtype=torch.float32)
        near(got, want, size, 1.0, 1e-6 + 0 * want, "scale %g" % scale)
    norm = float(torch.linalg.vector_norm(g))
    want = exact(g, steps=1, eps=norm)
    got = orthogonalize(g, steps=1, eps=norm, out_dtype=torch.float32)
    near(got, want, float(torch.linalg.vector_norm(want)), 1.0, 1e-6 + 0 * want, "eps")


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("rank,steps,coefficients", [(1, 3, ortho.COEFFICIENTS), (1, 5, ortho.COEFFICIENTS),
                                                     (5, 8, ortho.COEFFICIENTS), (None, 4, (2.0, -1.5, 0.5)),
                                                     (1, 6, (1.5, -0.5, 0.0))])
def test_joined_first_steps(rank, steps, coefficients, turn):
    """Matrices of low rank, and coefficients other than the usual ones, against the oracle's model of the joined steps:
    model and kernel round the same numbers, so that their errors are draws of one size."""
    shape = JOINED[::-1] if turn else JOINED
    announce("ortho joined %s rank %s steps %d" % (shape, rank, steps))
    rng = np.random.default_rng([100, rank or 0, steps])
    v = rng.standard_normal(shape) if rank is None else rng.standard_normal((shape[0], rank)) @ rng.standard_normal((rank, shape[1]))
    v = v.astype(np.float32)
    kw = dict(steps=steps, coefficients=coefficients)
    want = ortho.orthogonalize_ref(v, **kw)
    size = np.linalg.norm(want)
    model = np.linalg.norm(ortho.orthogonalize_model(v, joined=True, **kw) - want)
    got = orthogonalize(torch.from_numpy(v).cuda(), out_dtype=torch.float32, **kw).double().cpu().numpy()
    assert np.linalg.norm(got - want) <= 2 * model + 2.0 ** -20 * size


@pytest.mark.parametrize("shape,most", [((40, 90), 1.5e-2), ((85, 2715), 1.5e-2), ((209, 309), 1.5e-2), (JOINED, 2.5e-2),
                                        ((7700, 1920), 2.5e-2)])
def test_constant_matrices(shape, most):
    """The documented worst: every entry of a square rounds the same way."""
    announce("ortho constant %s" % (shape,))
    s = 1.0
    for _ in range(5):
        s = A * s + B * s ** 3 + C * s ** 5
    want = s / (shape[0] * shape[1]) ** 0.5
    got = orthogonalize(torch.full(shape, -3.0, device="cuda"), out_dtype=torch.float32).double()
    assert float((got + want).abs().max()) <= most * want
