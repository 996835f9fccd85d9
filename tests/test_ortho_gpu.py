"""Orthogonalized updates and the Muon step on the GPU against the float64 oracle.

The result is held to the oracle's own model of the kernels' roundings: model and kernel round the same numbers to
float16, each up to the order of float32 sums, so their errors against the definition are draws of one size.  A result may
be twice as far off (in norm) as the model's is, and what rounding it to its own type adds.
"""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import (AdamWState, AdamWTensors, MuonTensors, adamw_step, fp8_gemm, fp8_quantize,
                                           layer_norm, layer_norm_grad, muon_step, orthogonalize)
from gpu_helpers import announce
from oracle import ortho
from test_ortho_host import weight_gradient

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gradient(rows, cols, seed, dtype=torch.float32, kind="weight"):
    """A gradient on the GPU and its values in float64."""
    rng = np.random.default_rng([seed, rows, cols])
    v = weight_gradient(rng, rows, cols, max(1, min(rows, cols) // 4)) if kind == "weight" else \
        rng.standard_normal((rows, cols)) if kind == "normal" else \
        rng.standard_normal((rows, 1)) @ rng.standard_normal((1, cols))
    g = torch.from_numpy(1e-3 * v).to(dtype).cuda()
    return g, g.double().cpu().numpy()


def check(got, g, what, **kw):
    want = ortho.orthogonalize_ref(g, **kw)
    size = np.linalg.norm(want)
    model = np.linalg.norm(ortho.orthogonalize_model(g, **kw) - want)
    # float32 sums, which the model leaves out: K 2^-24 of the sum of the sizes at most, here as part of the norm
    allowed = 2 * model + (HALF[got.dtype] + 2.0 ** -20) * size
    off = np.linalg.norm(got.double().cpu().numpy() - want)
    assert off <= allowed, "%s: off by %g of the norm, allowed %g" % (what, off / size, allowed / size)


SHAPES = [(1, 1), (1, 5), (7, 1), (3, 2), (16, 16), (64, 64), (65, 64), (63, 130), (128, 256), (200, 70), (129, 1000),
          (777, 300), (256, 4096), (1000, 1000), (1403, 777), (40, 9000)]


@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape):
    for dtype, out in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        announce("ortho %s %s -> %s" % (shape, dtype, out))
        g, v = gradient(*shape, 1, dtype)
        got = orthogonalize(g, out_dtype=out)
        assert got.shape == g.shape and got.dtype == out
        check(got, v, shape)


@pytest.mark.parametrize("kind", ["weight", "normal", "rank 1"])
@pytest.mark.parametrize("steps,coefficients", [(1, ortho.COEFFICIENTS), (2, ortho.COEFFICIENTS), (5, ortho.COEFFICIENTS),
                                                (8, ortho.COEFFICIENTS), (7, (2.0, -1.5, 0.5)), (6, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(kind, steps, coefficients):
    announce("ortho steps %d %s %s" % (steps, coefficients, kind))
    for shape in ((300, 180), (100, 400)):
        g, v = gradient(*shape, 2, kind=kind)
        check(orthogonalize(g, steps=steps, coefficients=coefficients, out_dtype=torch.float32), v, shape, steps=steps,
              coefficients=coefficients)


@pytest.mark.parametrize("shapes", [[(1403, 777), (999, 2047), (2500, 1001), (333, 1500)], [(2304, 2100)],
                                    [(1600, 2100), (2100, 1600)], [(512, 512)] * 40, [(64, 64), (0, 8), (8, 0), (100, 3)]])
def test_lists(shapes):
    """Matrices worked on together, large enough for every tile; more of them than one launch takes; empty ones."""
    announce("ortho list %s" % shapes[:4])
    pairs = [gradient(*s, 10 + i) for i, s in enumerate(shapes)]
    got = orthogonalize([g for g, _ in pairs])
    for i, (o, (g, v)) in enumerate(zip(got, pairs)):
        assert o.shape == g.shape
        if v.size and (i < 3 or i == len(pairs) - 1):
            check(o, v, shapes[i])
    again = orthogonalize([g for g, _ in pairs])
    assert all(torch.equal(a, b) for a, b in zip(got, again))


SMALL = [(128, 256), (256, 128), (64, 512), (512, 64), (100, 250), (500, 17), (1, 512), (512, 1), (1, 513), (128, 192), (5, 3)]


@pytest.mark.parametrize("shapes", [[s] for s in SMALL] + [SMALL, SMALL * 4, SMALL + [(129, 64)], [(64, 64), (500, 300)]])
def test_small_matrices(shapes):
    """Matrices that one workgroup takes whole, alone, together, more than a launch's, and beside one that is larger."""
    announce("ortho small %s" % shapes[:3])
    pairs = [gradient(*s, 20 + i, torch.bfloat16 if i % 2 else torch.float32) for i, s in enumerate(shapes)]
    got = orthogonalize([g for g, _ in pairs], out_dtype=torch.float32)
    for o, (g, v), shape in zip(got, pairs, shapes):
        check(o, v, shape)
    assert all(torch.equal(a, b) for a, b in zip(got, orthogonalize([g for g, _ in pairs], out_dtype=torch.float32)))


def test_large_against_float64_on_the_gpu():
    """A square matrix of a large layer, and a wide one: every tile and a whole round of the chip."""
    for rows, cols in ((4096, 4096), (2048, 7936), (6016, 1920)):
        announce("ortho large %d x %d" % (rows, cols))
        gen = torch.Generator(device="cuda").manual_seed(rows)
        left = torch.randn((rows, 32), generator=gen, device="cuda") / torch.arange(1, 33, device="cuda")
        g = left @ torch.randn((32, cols), generator=gen, device="cuda")
        g += 0.1 * torch.randn((rows, cols), generator=gen, device="cuda")
        x = g.double()
        x /= torch.linalg.vector_norm(x) + 1e-7
        a, b, c = ortho.COEFFICIENTS
        for _ in range(5):
            if rows <= cols:
                s = x @ x.t().contiguous()
                x = a * x + (b * s + c * (s @ s)) @ x
            else:
                s = x.t().contiguous() @ x
                x = a * x + x @ (b * s + c * (s @ s))
        got = orthogonalize(g, out_dtype=torch.float32).double()
        # the documented bound
        assert float(torch.linalg.vector_norm(got - x)) <= 2e-3 * float(torch.linalg.vector_norm(x))
        # and no single tile astray: 64 x 64 pieces, whose errors are means of 4096 draws of one size
        d = (got - x).square().unfold(0, 64, 64).unfold(1, 64, 64).sum(dim=(2, 3))
        w = x.square().unfold(0, 64, 64).unfold(1, 64, 64).sum(dim=(2, 3))
        assert float((d / w).max()) <= (4 * 2e-3) ** 2


def test_views_and_what_lies_around_them():
    announce("ortho views")
    g, v = gradient(70, 90, 3)
    want = orthogonalize(g)
    buf = torch.full((80, 120), 7.0, device="cuda")
    src = buf[3:73, 5:95]
    src.copy_(g)
    dst = torch.full((80, 121), 5.0, dtype=torch.bfloat16, device="cuda")
    out = dst[2:72, 7:97]
    version = out._version
    assert orthogonalize(src, out=out) is out and out._version > version
    assert torch.equal(out, want)
    out.fill_(5.0)
    assert bool((dst == 5.0).all())
    src.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_special_values():
    announce("ortho special")
    z = torch.zeros(100, 64, device="cuda")
    assert not orthogonalize(z).any()
    for bad in (float("nan"), float("inf")):
        g, _ = gradient(100, 64, 4)
        good = g.clone()
        g[99, 63] = bad
        a, b = orthogonalize([g, good])
        assert a.isnan().all() and b.isfinite().all()
    # sums of squares outside float32's range: the scale of a gradient does not matter, far from eps
    g, v = gradient(64, 96, 5)
    want = orthogonalize(g, out_dtype=torch.float32)
    for scale in (2.0 ** 100, 2.0 ** -80):
        got = orthogonalize(g * scale, eps=1e-38, out_dtype=torch.float32)
        check(got, v, "scale %g" % scale, eps=1e-30)
    # eps as large as the norm halves the start
    norm = float(np.linalg.norm(v))
    check(orthogonalize(g, steps=1, eps=norm), v, "eps", steps=1, eps=norm)


def test_streams_and_graphs():
    """On another stream, and in a graph that replays with other gradients between eager work."""
    announce("ortho graph")
    pairs = [gradient(*s, 6) for s in ((300, 500), (700, 128))]
    gs = [g for g, _ in pairs]
    want = orthogonalize(gs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = orthogonalize(gs)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = orthogonalize(gs)
    for k in range(4):
        for i, (g, v) in enumerate(pairs):
            g.copy_(torch.from_numpy(np.roll(v, k, axis=0)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, orthogonalize(gs)))


def test_two_calls_at_once():
    """Two streams, and two captured graphs replayed on them, each with its own workspace: small, middle and large."""
    announce("ortho two at once")
    sets = [[gradient(*s, 30 + k)[0] for s in ((300, 500), (1024, 900))] + [gradient(128, 256, 40 + k)[0]]
            for k in range(2)]
    want = [[orthogonalize(g) for g in gs] for gs in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            got[k] = [orthogonalize(g) for _ in range(3) for g in sets[k]][-3:]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    graphs, outs = [], []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append([orthogonalize(g) for g in sets[k]])
        graphs.append(graph)
    for _ in range(3):
        for o in outs[0] + outs[1]:
            o.fill_(0.0)
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(outs, want) for a, b in zip(x, y))


def test_workspace_is_all_that_is_written():
    """The C entry with a workspace of exactly its size between guards, at sizes of every tile; twice on a workspace that
    holds NaN, so that nothing it held before comes through."""
    from block_scaled_fp4_hadamard_amd import _lib
    announce("ortho workspace")
    lib = _lib.lib()
    for shapes in ([(128, 256)], [(300, 180)], [(2048, 1990)], [(1000, 2900), (2900, 1000)], [(4096, 4160)]):
        gs = [gradient(*s, 50, torch.bfloat16)[0] if s[0] < 4000 else torch.randn(s, device="cuda").bfloat16()
              for s in shapes]
        outs = [torch.empty_like(g) for g in gs]
        array = (_lib.OrthoMatrixC * len(gs))(*[
            _lib.OrthoMatrixC(g.data_ptr(), o.data_ptr(), *g.shape, g.shape[1], g.shape[1], 1, 1)
            for g, o in zip(gs, outs)])
        size = lib.mx_orthogonalize_workspace(array, len(gs))
        buf = torch.full((size + 8192,), 255, dtype=torch.uint8, device="cuda")        # float16 NaN everywhere
        args = (array, len(gs), _lib.OrthoParamsC(3.4445, -4.7750, 2.0315, 1e-7, 5), buf.data_ptr() + 4096, size, None)
        torch.cuda.synchronize()
        assert lib.mx_orthogonalize(*args) == 0
        torch.cuda.synchronize()
        assert bool((buf[:4096] == 255).all()) and bool((buf[4096 + size:] == 255).all())
        assert all(torch.equal(o, w) for o, w in zip(outs, orthogonalize(gs)))
        del buf


# ---- the Muon step


def tensors_of(shapes, seed, dtype=torch.float32, copies=True):
    out = {k: [] for k in ("w", "g", "m", "h")}
    for i, (rows, cols) in enumerate(shapes):
        rng = np.random.default_rng([seed, i])
        out["w"].append(torch.from_numpy((0.02 * rng.standard_normal((rows, cols))).astype(np.float32)).cuda())
        out["g"].append(torch.from_numpy(1e-3 * weight_gradient(rng, rows, cols, 8)).to(dtype).cuda())
        out["m"].append(torch.from_numpy((1e-3 * weight_gradient(rng, rows, cols, 8)).astype(np.float32)).cuda())
        out["h"].append(torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda") if copies else None)
    return out


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("adjust", ["rms", "shape", "plain"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_muon_step(dtype, adjust, nesterov):
    for shapes in ([(200, 130), (64, 300), (65, 65), (1, 9), (300, 2)], [(128, 256), (200, 70), (65, 65), (1, 9), (300, 2)]):
        announce("muon %s %s %s %s" % (dtype, adjust, nesterov, shapes))
        one_step(shapes, dtype, adjust, nesterov)


def one_step(shapes, dtype, adjust, nesterov):
    t = tensors_of(shapes, 7, dtype, copies=adjust != "plain")
    before = [[x.double().cpu().numpy() for x in t[k]] for k in "wgm"]
    scale = torch.tensor([0.5], device="cuda") if adjust == "shape" else None
    lr = 0.02
    muon_step(MuonTensors(t["w"], t["g"], t["m"], copies=t["h"] if adjust != "plain" else None), lr=lr, momentum=0.9,
              weight_decay=0.2, nesterov=nesterov, adjust=adjust, grad_scale=scale)
    for i, (w, g, m) in enumerate(zip(*before)):
        s = 0.5 if scale is not None else 1.0
        ww, wm, o = ortho.muon_ref(w, g, m, lr, 0.9, 0.2, nesterov, adjust=adjust, scale=s)
        # m: momentum as a float32, two products and a sum: four roundings of their sizes
        tol = 4 * 2.0 ** -24 * (np.abs(m) * 0.9 + np.abs(g) * s * 0.1)
        assert np.all(np.abs(t["m"][i].double().cpu().numpy() - wm) <= tol)
        # w: the update's error in norm as check() has it, and its own roundings
        u = (g * s * 0.1 + wm * 0.9) if nesterov else wm
        rate = lr * ortho.adjust_of(w.shape, adjust)
        model = np.linalg.norm(ortho.orthogonalize_model(u) - o)
        got = t["w"][i].double().cpu().numpy()
        allowed = rate * (2 * model + 2.0 ** -20 * np.linalg.norm(o)) + \
            3 * 2.0 ** -24 * (np.linalg.norm(w) + rate * np.linalg.norm(o))
        assert np.linalg.norm(got - ww) <= allowed, (shapes[i], np.linalg.norm(got - ww), allowed)
        if adjust != "plain":
            assert torch.equal(t["h"][i], t["w"][i].bfloat16())


def test_muon_graph_with_a_rate_that_moves_on():
    announce("muon graph")
    shapes = [(200, 130), (130, 512), (64, 64)]
    a, b = tensors_of(shapes, 8), tensors_of(shapes, 8)
    lists = [MuonTensors(t["w"], t["g"], t["m"], copies=t["h"]) for t in (a, b)]
    lr, scale = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        muon_step(lists[0], lr=lr, grad_scale=scale)
    for k in range(4):
        rate = np.float32(1e-2 / (k + 1))
        lr.fill_(float(rate))
        scale.fill_(1.0 + k)
        graph.replay()
        torch.cuda.synchronize()
        muon_step(lists[1], lr=float(rate), grad_scale=scale)
        for key in ("w", "m", "h"):
            assert all(torch.equal(x, y) for x, y in zip(a[key], b[key]))


def test_muon_tells_autograd():
    w = torch.randn(64, 64, device="cuda", requires_grad=True)
    loss = (w * w).sum()
    t = MuonTensors([w.detach()], [torch.ones(64, 64, device="cuda")], [torch.zeros(64, 64, device="cuda")])
    muon_step(t, lr=1e-2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_a_layer_with_its_norm():
    """A linear behind a norm, trained as the operators are meant to be used together: norm, 8-bit cast and product, the
    gradients of both, Muon for the matrix and AdamW for the norm's vectors.  The norm's gradients are held to
    differences of the loss that the 8-bit product's own gradient defines."""
    announce("layer with norm")
    tokens, cin, cout = 512, 384, 640
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((tokens, cin), generator=gen, device="cuda").bfloat16()
    target = torch.randn((tokens, cout), generator=gen, device="cuda")
    weight, bias = torch.ones(cin, device="cuda"), torch.zeros(cin, device="cuda")
    master = 0.05 * torch.randn((cout, cin), generator=gen, device="cuda")
    copy, dw = master.bfloat16(), torch.empty_like(master)
    muon = MuonTensors([master], [dw], [torch.zeros_like(master)], copies=[copy])
    states = [AdamWState.zeros_like(v) for v in (weight, bias)]
    for step in range(1, 4):
        before = [v.clone() for v in (master, weight, bias)]
        y, mean, rstd = layer_norm(x, weight, bias)
        qy = fp8_quantize(y, axis="both")
        qw = fp8_quantize(copy, axis="both", kind="tile")
        out = fp8_gemm(qy["row"], qw["row"])
        dout = ((out - target) / tokens).bfloat16()
        qd = fp8_quantize(dout, axis="both", fmt="e5m2")
        dy = fp8_gemm(qd["row"], qw["col"], out_dtype=torch.bfloat16)
        fp8_gemm(qd["col"], qy["col"], out=dw)
        dx, dweight, dbias = layer_norm_grad(dy, x, mean, rstd, weight)
        muon_step(muon, lr=1e-2)
        adamw_step(AdamWTensors([weight, bias], [dweight, dbias], states), lr=1e-2, step=step)
        assert dx.isfinite().all() and torch.equal(copy, master.bfloat16())
        assert all(not torch.equal(a, b) for a, b in zip((master, weight, bias), before))
        # the norm's part of the chain, in float64 by differences: L(w, b) = sum(dy * y(w, b))
        x64, d64 = x.double(), dy.double()
        for vec, grad, which in ((before[1], dweight, 0), (before[2], dbias, 1)):
            at = int(grad.abs().argmax())
            loss = []
            for sign in (1, -1):
                p = [before[1].double(), before[2].double()]
                p[which][at] += sign * 1e-3
                h = x64 - x64.mean(dim=1, keepdim=True)
                h = h / (h.square().mean(dim=1, keepdim=True) + 1e-5).sqrt()
                loss.append(float((d64 * (h * p[0] + p[1])).sum()))
            # linear in the vector: differences are exact up to float64, the kernel up to float32's sums
            size = float((d64[:, at].abs() * (h[:, at].abs() if which == 0 else 1.0)).sum())
            assert abs((loss[0] - loss[1]) / 2e-3 - float(grad[at])) <= 300 * 2.0 ** -24 * size + 1e-9


@pytest.mark.parametrize("shape", [(100, 64), (300, 200)])
def test_zeros_stay_zeros_with_any_eps(shape):
    """One workgroup's kernel and the tiles', down to the smallest double."""
    announce("ortho zeros %s" % (shape,))
    for eps in (1e-7, 1e-300, 1e-306, 5e-324):
        assert not orthogonalize(torch.zeros(shape, device="cuda"), eps=eps, out_dtype=torch.float32).any()
    w = torch.ones(shape, device="cuda")
    z = torch.zeros_like(w)
    muon_step(MuonTensors([w], [z], [z.clone()]), lr=0.5, weight_decay=0.0, eps=1e-306)
    assert torch.equal(w, torch.ones_like(w))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(64, 96), (300, 200), (200, 300)])
def test_subnormal_gradients(shape, dtype):
    """Whole multiples of the type's smallest number are as good a gradient as any."""
    announce("ortho subnormal %s %s" % (shape, dtype))
    rng = np.random.default_rng([60, *shape])
    v = rng.integers(1, 64, shape) * np.sign(rng.standard_normal(shape)) * torch.finfo(dtype).smallest_normal * \
        torch.finfo(dtype).eps
    g = torch.from_numpy(v).to(dtype).cuda()
    assert np.array_equal(g.double().cpu().numpy(), v)
    check(orthogonalize(g, eps=1e-60, out_dtype=torch.float32), v, "subnormal %s" % (shape,), eps=1e-60)
