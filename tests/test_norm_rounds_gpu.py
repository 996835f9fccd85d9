"""Norms of more rows than the resident workgroups take at once, through every kernel, both kinds and both types; and the
C entries' sums one at a time.  The reference is the formula in float64 on the GPU."""
import pytest
import torch

from block_scaled_fp4_hadamard_amd import _lib, layer_norm, layer_norm_grad
from gpu_helpers import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24            # half a float32 step, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}

# (rows, columns): a row of 16, 64, 256 and 1024 lanes or 512 with sums in LDS, and rows wider than a workgroup's
# registers.  2048 workgroups of 16, 4 or 1 rows, or 512 of one, are a round forward; 256 of 64, 16, 4 or 1 backward.  The
# last round is part-filled, and no width is a whole number of vectors.
SHAPES = {
    torch.float32: [(40001, 59), (40001, 99), (17001, 250), (17001, 501), (9001, 599), (5001, 1001), (4501, 2001),
                    (2501, 4001), (2101, 5003), (2101, 7001), (1301, 9001), (1301, 14335), (1301, 18001),
                    (1301, 20001)],
    torch.bfloat16: [(40001, 99), (40001, 199), (17001, 401), (9001, 901), (9001, 1499), (5001, 1999), (4501, 4001),
                     (2101, 6001), (2101, 9001), (2101, 15001), (1301, 17001), (1301, 20001), (1301, 33001)],
}


def depth(cols):
    """Additions on the longest way through a row's sum: a lane's own elements (at most 64 in registers, every 1024th of
    wider rows, whole vectors), the lanes, the waves; four more for the operations on each element."""
    return max(64, -(-cols // 1024) + 8) + 6 + 16 + 4


def case(rows, cols, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000 * seed + rows + cols)
    x = torch.randn((rows, cols), generator=gen, device="cuda") + 0.3
    dy = 1e-3 * torch.randn((rows, cols), generator=gen, device="cuda")
    hot = torch.rand((1, cols), generator=gen, device="cuda") < 0.02
    w = 1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    b = torch.randn(cols, generator=gen, device="cuda")
    return [t.to(dtype) for t in (torch.where(hot, 30 * x, x), torch.where(hot, 30 * dy, dy), w, b)]


def within(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), "%s: %d of %d outside, first at %s, worst %g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float((off / tol.clamp_min(1e-300)).max()))


def check_forward(x, w, b, kind, got, eps=1e-5):
    y, mean, rstd = got
    v, ww = x.double(), w.double()
    n = depth(x.shape[1]) * U
    size = v.abs().mean(dim=1)
    wm = v.mean(dim=1) if kind == "layer" else torch.zeros_like(size)
    d = v - wm[:, None]
    var = d.square().mean(dim=1)
    wr = (var + eps).rsqrt()
    # a sum of float32 numbers is off by n of the sum of their sizes
    mean_off = n * size if kind == "layer" else 0 * size
    if kind == "layer":
        within(mean, wm, mean_off, "mean")
    else:
        assert mean is None
    # the mean's error moves the variance by its square; d's rounding, U (|x| + |mean|), by 2 |d| times that, which
    # Cauchy-Schwarz bounds by 2 U rms(d) (rms(x) + |mean|); and the sum's own
    off = mean_off.square() + n * var + 2 * U * var.sqrt() * (v.square().mean(dim=1).sqrt() + wm.abs())
    rel = off / (var + eps) + 4 * U
    within(rstd, wr, rel * wr, "rstd")
    hw = d * wr[:, None] * ww
    want = hw + b.double() if b is not None else hw
    tol = ww.abs() * wr[:, None] * (mean_off[:, None] + U * (d.abs() + wm.abs()[:, None])) * 1.01 + \
        (rel[:, None] + 3 * U) * hw.abs() + U * want.abs()
    within(y, want, tol + HALF[x.dtype] * (want.abs() + tol), "y")


def check_backward(dy, x, w, kind, mean, rstd, got):
    dx, dw, db = got
    rows, cols = x.shape
    d, ww, r = dy.double(), w.double(), rstd.double()[:, None]
    h = (x.double() - (mean.double()[:, None] if mean is not None else 0.0)) * r
    g = d * ww
    want = g - h * (g * h).mean(dim=1, keepdim=True)
    inner = g.abs() + h.abs() * (g * h).abs().mean(dim=1, keepdim=True)
    if kind == "layer":
        want = want - g.mean(dim=1, keepdim=True)
        inner = inner + g.abs().mean(dim=1, keepdim=True)
    want = want * r
    # h carries two roundings, of the difference and of the product, g one
    tol = (depth(cols) + 8) * U * inner * r
    within(dx, want, tol + HALF[x.dtype] * (want.abs() + tol), "dx")
    # over the rows: a lane's own, the workgroup's (64 at most), the workgroups' (16 + 16), h's and the product's roundings
    n = (-(-rows // 256) + 64 + 32 + 4) * U
    within(dw, (d * h).sum(dim=0), n * (d * h).abs().sum(dim=0), "dweight")
    if kind == "layer":
        within(db, d.sum(dim=0), n * d.abs().sum(dim=0), "dbias")
    else:
        assert db is None


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,shape", [(t, s) for t in SHAPES for s in SHAPES[t]])
def test_several_rounds_of_every_kernel(dtype, shape, kind):
    announce("norm rounds %s %s %s" % (dtype, shape, kind))
    x, dy, w, b = case(*shape, dtype, 1)
    b = b if kind == "layer" else None
    got = layer_norm(x, w, b, kind=kind)
    check_forward(x, w, b, kind, got)
    back = layer_norm_grad(dy, x, got[1], got[2], w, kind=kind)
    check_backward(dy, x, w, kind, got[1], got[2], back)
    again = layer_norm(x, w, b, kind=kind) + layer_norm_grad(dy, x, got[1], got[2], w, kind=kind)
    assert all(p is q is None or torch.equal(p, q) for p, q in zip(got + back, again))


def entry(x, dy, w, mean, rstd, kind, dw, db):
    """dx and the sums that are asked for, of the C entry, on a workspace that holds NaN."""
    lib = _lib.lib()
    rows, cols = x.shape
    type_ = {torch.float32: 0, torch.bfloat16: 1}[x.dtype]
    size = lib.mx_layer_norm_grad_workspace(rows, cols, type_, dw is not None or db is not None)
    space = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    torch.cuda.synchronize()
    st = lib.mx_layer_norm_grad(dy.data_ptr(), cols, x.data_ptr(), cols, type_, rows, cols, w.data_ptr(), type_,
                                None if mean is None else mean.data_ptr(), rstd.data_ptr(), kind, dx.data_ptr(), cols,
                                None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(),
                                space.data_ptr() if size else None, size, None)
    torch.cuda.synchronize()
    assert st == 0
    return dx


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(33, 500), (2501, 1499), (300, 15001), (300, 33001)])
def test_sums_one_at_a_time(dtype, shape):
    """Either sum alone is the one of both, and dbias comes for RMS rows too."""
    announce("norm sums %s %s" % (dtype, shape))
    x, dy, w, b = case(*shape, dtype, 2)
    cols = shape[1]
    _, mean, rstd = layer_norm(x, w, b)
    dx, dw, db = layer_norm_grad(dy, x, mean, rstd, w)
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        gw, gb = (torch.full((cols,), -1.0, device="cuda") for _ in range(2))
        assert torch.equal(entry(x, dy, w, mean, rstd, 0, gw if want_w else None, gb if want_b else None), dx)
        assert torch.equal(gw, dw if want_w else torch.full_like(gw, -1.0))
        assert torch.equal(gb, db if want_b else torch.full_like(gb, -1.0))
    _, _, rstd = layer_norm(x, w, kind="rms")
    dx, dw, _ = layer_norm_grad(dy, x, None, rstd, w, kind="rms")
    gw, gb = (torch.empty(cols, device="cuda") for _ in range(2))
    assert torch.equal(entry(x, dy, w, None, rstd, 1, gw, gb), dx) and torch.equal(gw, dw)
    # dbias does not depend on the statistics
    assert torch.equal(gb, db)


@pytest.mark.parametrize("cols", [300, 4000, 40000])
def test_statistics_are_optional(cols):
    announce("norm without statistics %d" % cols)
    x, _, w, b = case(70, cols, torch.bfloat16, 3)
    for kind, bias in (("layer", b), ("rms", None)):
        want = layer_norm(x, w, bias, kind=kind)[0]
        y = torch.empty_like(x)
        torch.cuda.synchronize()
        st = _lib.lib().mx_layer_norm(x.data_ptr(), 1, 70, cols, cols, w.data_ptr(), None if bias is None else b.data_ptr(),
                                      1, 1e-5, _lib.NORM[kind], y.data_ptr(), cols, None, None, None)
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(y, want)
