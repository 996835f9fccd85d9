"""Layer norm, its RMS form and their backward pass on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import layer_norm, layer_norm_grad
from gpu_helpers import announce
from oracle import norm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24            # half a float32 step, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
# every layout of a row (16, 64, 256 and 1024 lanes, one to four vectors), its borders, and rows wider than a workgroup
WIDTHS = [1, 3, 8, 64, 127, 128, 129, 256, 257, 512, 516, 768, 1000, 1100, 1536, 1025, 2048, 4096, 4099, 8192, 8200, 16384, 16385, 33000]


def depth(cols):
    """Additions on the longest way through a row's sum: a lane's own elements (32, or every 1024th vector), the lanes,
    the waves; four more for the operations on each element."""
    return max(32, -(-cols // 1024)) + 6 + 16 + 4


def case(rows, cols, dtype, seed, pitch=0, offset=0):
    """x, dy on the GPU (views with a pitch, `offset` elements into their buffers) and their values in float64."""
    rng = np.random.default_rng([seed, rows, cols])
    out = []
    for k in range(2):
        v = rng.standard_normal((rows, cols)) * (1.0 if k == 0 else 1e-3) + (0.3 if k == 0 else 0.0)
        v[:, rng.random(cols) < 0.02] *= 30.0
        buf = torch.full((offset + rows * (cols + pitch) + 8,), 7.0, dtype=dtype, device="cuda")
        x = buf.as_strided((rows, cols), (cols + pitch, 1), offset)
        x.copy_(torch.from_numpy(v).to(dtype))
        out += [x, x.double().cpu().numpy()]
    return out


def weights(cols, dtype, seed):
    rng = np.random.default_rng([seed, cols])
    w, b = (torch.from_numpy(v).to(dtype).cuda() for v in (1 + 0.1 * rng.standard_normal(cols), rng.standard_normal(cols)))
    return w, b


def within(got, want, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %g of the tolerance" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))


def check_forward(x, vx, w, b, kind, got, eps=1e-5):
    y, mean, rstd = got
    f = [None if t is None else t.double().cpu().numpy() for t in (w, b)]
    wy, wm, wr = norm.forward_ref(vx, *f, eps=eps, kind=kind)
    n = depth(vx.shape[1]) * U
    size = np.abs(vx).mean(axis=1)                        # a sum of float32 numbers is off by n of the sum of their sizes
    if kind == "layer":
        within(mean, wm, n * size, "mean")
    else:
        assert mean is None
    # the mean's error moves the variance by its square; the rest is the roundings of d (relative to |x| + |mean|), d^2
    # and the sum: d's enter as 2 |d| U (|x| + |mean|), which Cauchy-Schwarz bounds by 2 U rms(d) (rms(x) + |mean|)
    d = vx - wm[:, None]
    var = (d * d).mean(axis=1)
    off = (n * size) ** 2 + n * var + \
        2 * U * np.sqrt(var) * (np.sqrt((vx * vx).mean(axis=1)) + np.abs(wm))
    rel = off / (var + eps) + 4 * U
    within(rstd, wr, rel * wr, "rstd")
    a = np.abs(wy - (0.0 if f[1] is None else f[1]))      # |h w|
    ww = 1.0 if f[0] is None else np.abs(f[0])
    mean_off = (n * size if kind == "layer" else 0 * size)[:, None]
    tol = ww * wr[:, None] * (mean_off + U * (np.abs(d) + np.abs(wm)[:, None])) * 1.01 + (rel[:, None] + 3 * U) * a + \
        U * np.abs(wy)
    half = HALF[x.dtype]
    within(y, wy, tol + half * (np.abs(wy) + tol), "y")


def check_backward(dy, vdy, x, vx, w, kind, mean, rstd, got):
    dx, dw, db = got
    rows, cols = vx.shape
    f = None if w is None else w.double().cpu().numpy()
    m = np.zeros(rows) if mean is None else mean.double().cpu().numpy()
    r = rstd.double().cpu().numpy()
    wx, ww, wb = norm.backward_ref(vdy, vx, m, r, f, kind)
    h = (vx - m[:, None]) * r[:, None]
    g = vdy if f is None else vdy * f
    n = depth(cols) * U
    # h carries two roundings (of the difference, relative to itself, and of the product), g one
    inner = np.abs(g) + np.abs(h) * np.abs(g * h).mean(axis=1)[:, None]
    if kind == "layer":
        inner = inner + np.abs(g).mean(axis=1)[:, None]
    tol = (n + 8 * U) * inner * r[:, None]
    within(dx, wx, tol + HALF[x.dtype] * (np.abs(wx) + tol), "dx")
    # over the rows: a lane's own (256 workgroups share them), the workgroup's (64 at most), the workgroups' (16 + 16)
    n = (-(-rows // 256) + 64 + 32 + 4) * U
    within(dw, ww, n * np.abs(vdy * h).sum(axis=0), "dweight")
    if kind == "layer":
        within(db, wb, n * np.abs(vdy).sum(axis=0), "dbias")
    else:
        assert db is None


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_rows_of_every_width(cols, dtype, kind):
    for rows, pitch, offset in ((1, 0, 0), (67, 5, 3)):
        announce("norm %d x %d %s %s pitch %d offset %d" % (rows, cols, dtype, kind, pitch, offset))
        x, vx, dy, vdy = case(rows, cols, dtype, 1, pitch, offset)
        w, b = weights(cols, dtype if rows == 1 else torch.float32, 2)
        if kind == "rms":
            b = None
        got = layer_norm(x, w, b, kind=kind)
        check_forward(x, vx, w, b, kind, got)
        back = layer_norm_grad(dy, x, got[1], got[2], w, kind=kind)
        check_backward(dy, vdy, x, vx, w, kind, got[1], got[2], back)


@pytest.mark.parametrize("rows,cols", [(5000, 64), (20001, 128), (3000, 512), (3001, 600), (4097, 1024), (2001, 4096), (1500, 9001)])
def test_many_rows(rows, cols):
    """More rows than the resident workgroups take at once, the last round part-filled."""
    announce("norm rows %d x %d" % (rows, cols))
    x, vx, dy, vdy = case(rows, cols, torch.bfloat16, 3)
    w, b = weights(cols, torch.bfloat16, 4)
    got = layer_norm(x, w, b)
    check_forward(x, vx, w, b, "layer", got)
    back = layer_norm_grad(dy, x, got[1], got[2], w)
    check_backward(dy, vdy, x, vx, w, "layer", got[1], got[2], back)
    again = layer_norm_grad(dy, x, got[1], got[2], w)
    assert all(torch.equal(p, q) for p, q in zip(back, again))


@pytest.mark.parametrize("cols", [100, 4096, 20000])
def test_without_weight_and_mixed_types(cols):
    announce("norm plain %d" % cols)
    x, vx, dy, vdy = case(9, cols, torch.float32, 5)
    w, b = weights(cols, torch.bfloat16, 6)
    for ww, bb in ((None, None), (w, None), (None, b)):
        got = layer_norm(x, ww, bb)
        check_forward(x, vx, ww, bb, "layer", got)
        check_backward(dy, vdy, x, vx, ww, "layer", got[1], got[2], layer_norm_grad(dy, x, got[1], got[2], ww))
    dx, dw, db = layer_norm_grad(dy, x, got[1], got[2], sums=False)
    assert dw is None and db is None and torch.equal(dx, layer_norm_grad(dy, x, got[1], got[2])[0])


def test_outputs_in_place_of_new_ones_and_what_lies_around_them():
    announce("norm out")
    x, vx, dy, vdy = case(33, 1001, torch.bfloat16, 7, pitch=7)
    w, b = weights(1001, torch.float32, 8)
    y, mean, rstd = layer_norm(x, w, b)
    dx, dw, db = layer_norm_grad(dy, x, mean, rstd, w)
    for want, call in ((y, lambda o: layer_norm(x, w, b, out=o)[0]),
                       (dx, lambda o: layer_norm_grad(dy, x, mean, rstd, w, out=o)[0])):
        buf = torch.full((36, 1020), 5.0, dtype=torch.bfloat16, device="cuda")
        out = buf[1:34, 3:1004]
        version = out._version
        assert call(out) is out and out._version > version
        assert torch.equal(out, want)
        buf[1:34, 3:1004] = 5.0
        assert bool((buf == 5.0).all())


def test_empty():
    for shape in ((0, 64), (5, 0), (0, 0)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        y, mean, rstd = layer_norm(x)
        dx, dw, db = layer_norm_grad(x, x, mean, rstd)
        assert y.shape == dx.shape == x.shape and dw.shape == db.shape == (shape[1],)
        assert not dw.any() and not db.any()         # no rows: the sums are zero


def test_rows_that_are_special():
    """NaN and Inf stay in their rows, a constant row becomes the bias, and the sums over rows take them in."""
    announce("norm special")
    x, vx, dy, vdy = case(6, 300, torch.float32, 9)
    w, b = weights(300, torch.float32, 10)
    clean = layer_norm(x, w, b)[0]
    x[1, 7], x[2, 299], x[3] = float("nan"), float("inf"), 4.0
    y, mean, rstd = layer_norm(x, w, b)
    assert y[1].isnan().all() and y[2].isnan().all() and torch.equal(y[3], b)
    assert torch.equal(y[[0, 4, 5]], clean[[0, 4, 5]])
    assert rstd[3].item() == pytest.approx(1e-5 ** -0.5, rel=1e-6)
    dx, dw, db = layer_norm_grad(dy, x, mean, rstd, w)
    assert dx[1].isnan().all() and dx[2].isnan().all() and dx[[0, 3, 4, 5]].isfinite().all()
    assert dw.isnan().all() and db.isfinite().all()
    y, _, rstd = layer_norm(x, w, kind="rms")
    assert y[1].isnan().all() and rstd[2].item() == 0.0 and y[2, 299].isnan() and not y[2, :299].any()
    assert layer_norm(torch.zeros(2, 8, device="cuda"), eps=0.0, kind="rms")[0].isnan().all()
    # values whose float32 difference to a large mean is exact: the variance has no cancellation left in it
    far = torch.full((1, 256), 65536.0, device="cuda")
    far[0, ::2] += 1.0
    y, mean, rstd = layer_norm(far, eps=0.0)
    assert mean.item() == 65536.5 and rstd.item() == 2.0 and torch.equal(y.abs(), torch.ones_like(y))


def test_offsets_past_32_bits():
    """The last rows of a matrix of over 4 GiB."""
    announce("norm large")
    rows, cols = (1 << 32) // 2 // 4096 + 3, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail, vt, _, _ = case(4, cols, torch.bfloat16, 11)
    x[-4:] = tail
    y, mean, rstd = layer_norm(x)
    check_forward(tail, vt, None, None, "layer", (y[-4:], mean[-4:], rstd[-4:]))
    dy = y                                   # any gradient does
    dx, dw, db = layer_norm_grad(dy, x, mean, rstd)
    want = layer_norm_grad(dy[-4:].contiguous(), tail, mean[-4:], rstd[-4:])
    assert torch.equal(dx[-4:], want[0])
    # all other rows are zeros: their y, hence dy, is zero, and four terms are added in either order
    h = (tail.double() - mean[-4:, None].double()) * rstd[-4:, None].double()
    for got, ref, size in ((dw, want[1], (y[-4:].double() * h).abs().sum(dim=0)),
                           (db, want[2], y[-4:].double().abs().sum(dim=0))):
        assert bool(((got.double() - ref.double()).abs() <= 8 * U * size).all())


def test_on_another_stream_and_in_a_graph():
    announce("norm graph")
    x, vx, dy, vdy = case(65, 4096, torch.bfloat16, 12)
    w, b = weights(4096, torch.bfloat16, 13)

    def both():
        y, mean, rstd = layer_norm(x, w, b)
        return (y, mean, rstd) + layer_norm_grad(dy, x, mean, rstd, w)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in range(4):
        x.copy_(torch.from_numpy(vx * (1 + k)).to(x.dtype))
        for t in got:
            t.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = both()
        assert all(torch.equal(p, q) for p, q in zip(got, eager))


def test_two_calls_at_once():
    """Two streams at once, each call with its own workspace."""
    announce("norm two at once")
    sets = [case(700, cols, torch.bfloat16, 14 + k) for k, cols in enumerate((4096, 17000))]
    want = [layer_norm_grad(s[2], s[0], *layer_norm(s[0])[1:]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for s, stream in zip(sets, streams):
        with torch.cuda.stream(stream):
            got.append([layer_norm_grad(s[2], s[0], *layer_norm(s[0])[1:]) for _ in range(4)][-1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


@pytest.mark.parametrize("rows,cols,dtype", [(1, 1, torch.float32), (300, 4096, torch.bfloat16), (5, 14000, torch.float32),
                                             (260, 19456, torch.bfloat16), (3, 19457, torch.float32)])
def test_workspace_is_all_that_is_written(rows, cols, dtype):
    """The C entry with a workspace of exactly its size between guards."""
    from block_scaled_fp4_hadamard_amd import _lib
    announce("norm workspace %d x %d" % (rows, cols))
    lib = _lib.lib()
    x, _, dy, _ = case(rows, cols, dtype, 16)
    _, mean, rstd = layer_norm(x)
    kind = 0 if dtype == torch.float32 else 1
    size = lib.mx_layer_norm_grad_workspace(rows, cols, kind, 1)
    buf = torch.full((size + 8192,), 255, dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    torch.cuda.synchronize()
    st = lib.mx_layer_norm_grad(dy.data_ptr(), cols, x.data_ptr(), cols, kind, rows, cols, None, 0, mean.data_ptr(),
                                rstd.data_ptr(), 0, dx.data_ptr(), cols, dw.data_ptr(), db.data_ptr(),
                                buf.data_ptr() + 4096, size, None)
    torch.cuda.synchronize()
    assert st == 0 and bool((buf[:4096] == 255).all()) and bool((buf[4096 + size:] == 255).all())
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), layer_norm_grad(dy, x, mean, rstd)))


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_statistics_of_rows_without_columns(kind):
    """0 / 0, and not what the memory held before."""
    announce("norm stats of nothing %s" % kind)
    held = [torch.full((5,), 7.0, device="cuda") for _ in range(16)]
    del held
    for dtype in (torch.float32, torch.bfloat16):
        _, mean, rstd = layer_norm(torch.zeros((5, 0), dtype=dtype, device="cuda"), kind=kind)
        assert rstd.shape == (5,) and rstd.isnan().all()
        assert mean is None if kind == "rms" else mean.isnan().all()


def test_gradient_of_more_columns_than_a_launch_has_lanes():
    """The sums of 2^28 columns and more.  Values of -1, 0 and 1 and statistics of 0 and 1: every sum is a whole number
    below 2^24, exact in any order, and dx is off by the roundings of its own four operations."""
    announce("norm grad of 2^28 columns")
    rows, cols = 2, (1 << 28) + 70
    gen = torch.Generator(device="cuda").manual_seed(17)
    x, dy = (torch.randint(-1, 2, (rows, cols), generator=gen, device="cuda", dtype=torch.int8).bfloat16() for _ in range(2))
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dx, dw, db = layer_norm_grad(dy, x, mean, rstd)
    step = 1 << 25
    runs = [slice(a, a + step) for a in range(0, cols, step)]
    c1, c2 = (sum(f(r) for r in runs) / cols for f in (lambda r: dy[:, r].double().sum(dim=1),
                                                       lambda r: (dy[:, r].double() * x[:, r].double()).sum(dim=1)))
    for r in runs:
        g, h = dy[:, r].double(), x[:, r].double()
        assert torch.equal(dw[r].double(), (g * h).sum(dim=0)) and torch.equal(db[r].double(), g.sum(dim=0))
        want = g - c1[:, None] - h * c2[:, None]
        tol = 4 * U * (g.abs() + c1.abs()[:, None] + h.abs() * c2.abs()[:, None])
        assert bool(((dx[:, r].double() - want).abs() <= tol + HALF[torch.bfloat16] * (want.abs() + tol)).all())
