"""Orthogonalized updates without a GPU: the oracle against singular values, the bounds of the iteration, every refusal,
and the list that a Muon step takes."""
import ctypes

import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import MuonTensors, _lib, muon_step, orthogonalize
from oracle import ortho

FAKE = 0x10000          # an aligned non-null address; validation never dereferences it
A, B, C = ortho.COEFFICIENTS


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (7, 7), (1, 30), (30, 1), (1, 1)])
def test_reference_acts_on_singular_values(shape):
    g = np.random.default_rng(1).standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(5):
        s = A * s + B * s ** 3 + C * s ** 5
    assert np.allclose(ortho.orthogonalize_ref(g), (u * s) @ vt, rtol=0, atol=1e-12)
    assert np.all((s > 0.3) & (s < 1.2))


def test_five_steps_take_singular_values_near_one():
    """What the documentation says of the usual coefficients, over all starts from 0.01 on."""
    s = np.linspace(0.01, 1.0, 100001)
    for _ in range(5):
        s = A * s + B * s ** 3 + C * s ** 5
    assert 0.67 < s.min() and s.max() < 1.14


def weight_gradient(rng, rows, cols, rank):
    strong = (rng.standard_normal((rows, rank)) / np.arange(1, rank + 1)) @ rng.standard_normal((rank, cols))
    return strong + 0.1 * rng.standard_normal((rows, cols))


def test_rounding_costs_less_than_bf16():
    """The documented 2e-3, on the hard kinds: random, few strong directions, rank 1."""
    rng = np.random.default_rng(2)
    for g in (rng.standard_normal((96, 96)), weight_gradient(rng, 128, 384, 16), rng.standard_normal((200, 1)) @
              rng.standard_normal((1, 100)), rng.standard_normal((64, 1000))):
        ref = ortho.orthogonalize_ref(g)
        assert np.linalg.norm(ortho.orthogonalize_model(g) - ref) <= 2e-3 * np.linalg.norm(ref)


# ---- refusals of the C entries


def matrix(g=FAKE, out=FAKE, rows=64, cols=32, ld_g=32, ld_out=32, grad=0, type=1):
    return _lib.OrthoMatrixC(g, out, rows, cols, ld_g, ld_out, grad, type)


def params(a=A, b=B, c=C, eps=1e-7, steps=5):
    return _lib.OrthoParamsC(a, b, c, eps, steps)


def call(items, count=None, p=None, ws=FAKE, bytes=1 << 40):
    array = (_lib.OrthoMatrixC * max(1, len(items)))(*items)
    return _lib.lib().mx_orthogonalize(array, len(items) if count is None else count, params() if p is None else p, ws,
                                       bytes, None)


@pytest.mark.parametrize("kw", [dict(g=None), dict(g=FAKE + 2), dict(g=FAKE + 1, grad=1), dict(out=None),
                                dict(out=FAKE + 1), dict(out=FAKE + 2, type=0), dict(rows=-1), dict(cols=-1),
                                dict(rows=1 << 20), dict(cols=1 << 20), dict(rows=1 << 16, cols=1 << 16, ld_g=1 << 16,
                                                                              ld_out=1 << 16),
                                dict(ld_g=31), dict(ld_out=31), dict(ld_out=1 << 26), dict(grad=2), dict(type=-1)])
def test_matrix_refusals(kw):
    assert call([matrix(rows=0), matrix(**kw)]) == 1


@pytest.mark.parametrize("kw", [dict(steps=0), dict(steps=65), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(a=float("nan")), dict(b=float("inf")), dict(a=5.0),
                                dict(a=3.0, b=0.0, c=0.0), dict(a=1.5, b=16.0, c=-14.0), dict(a=-4.1, b=0.0, c=0.0),
                                dict(a=1.0, b=-20.0, c=19.5), dict(a=1.0, b=1.0, c=1.0)])
def test_parameter_refusals(kw):
    assert call([matrix(rows=0)], p=params(**kw)) == 1


@pytest.mark.parametrize("kw", [{}, dict(steps=64), dict(steps=1, a=3.0, b=0.0, c=0.0), dict(a=1.5, b=-0.5, c=0.0),
                                dict(a=2.0, b=-1.5, c=0.5), dict(a=15.0 / 8, b=-10.0 / 8, c=3.0 / 8),
                                dict(a=0.0, b=0.0, c=0.0)])
def test_parameters_that_stay_bounded(kw):
    assert call([matrix(rows=0)], p=params(**kw)) == 0


def test_workspace_and_groups():
    ask = _lib.lib().mx_orthogonalize_workspace

    def need(*shapes):
        array = (_lib.OrthoMatrixC * max(1, len(shapes)))(*[matrix(rows=r, cols=c) for r, c in shapes])
        return ask(array, len(shapes))

    one = need((100, 300))
    # 100 and 300 in whole steps of 64, and 192 more for a tile's rest
    assert one == 8 * 256 + 2 * (3 * 320 * 512 + 3 * 320 * 320) == need((300, 100))
    assert need((100, 300), (0, 5), (100, 300)) == 2 * one
    assert need(*[(100, 300)] * 40) == 32 * one                     # 32 matrices are worked on at a time
    # and within 2 GiB
    assert need(*[(8192, 16384)] * 3) == need((8192, 16384)) > 1 << 30
    assert need(*[(6400, 15744)] * 3) == 2 * need((6400, 15744)) < 1 << 31
    assert need((40000, 60000)) > 1 << 33                          # but one matrix whatever its size
    assert need() == need((0, 3)) == need((1 << 20, 5)) == need((1 << 16, 1 << 16)) == need((-1, 5)) == 0
    assert ask(None, 3) == 0 and ask(None, -1) == 0
    assert call([matrix(rows=100, cols=300, ld_g=300, ld_out=300)], bytes=one - 1) == 1
    assert call([matrix()], ws=None) == call([matrix()], ws=FAKE + 8) == 1
    assert call([], ws=None, bytes=0) == call([matrix(rows=0, g=None, out=None)], ws=None, bytes=0) == 0
    assert call([], count=-1) == 1
    assert _lib.lib().mx_orthogonalize(None, 1, params(), FAKE, 1 << 40, None) == 1
    assert _lib.lib().mx_orthogonalize(None, 0, None, None, 0, None) == 1


def muon(tensor=None, count=1, ws=FAKE, bytes=1 << 40, ortho=None, lr=1e-3, momentum=0.9, decay=0.1, nesterov=1, adjust=1,
         lr_dev=None, scale=None, **kw):
    t = dict(w=FAKE, g=FAKE, m=FAKE, copy=FAKE, rows=64, cols=32, grad=0) | kw
    p = _lib.MuonParamsC(ortho or params(), lr, momentum, decay, nesterov, adjust, lr_dev, scale)
    return _lib.lib().mx_muon_step((_lib.MuonTensorC * 1)(_lib.MuonTensorC(**t)), count, p, ws, bytes, None)


@pytest.mark.parametrize("kw", [dict(count=-1), dict(ortho=params(steps=0)), dict(ortho=params(a=9.0)), dict(momentum=1.0),
                                dict(momentum=-0.1), dict(momentum=float("nan")), dict(momentum=1 - 2.0 ** -40),
                                dict(decay=float("inf")), dict(nesterov=2), dict(adjust=3), dict(lr=float("nan")),
                                dict(lr_dev=FAKE + 2), dict(scale=FAKE + 1), dict(w=None), dict(w=FAKE + 2), dict(g=None),
                                dict(g=FAKE + 2), dict(g=FAKE + 1, grad=1), dict(m=None), dict(m=FAKE + 2),
                                dict(copy=FAKE + 1), dict(rows=-1), dict(cols=1 << 20), dict(grad=2), dict(ws=None),
                                dict(ws=FAKE + 4), dict(bytes=10000)])
def test_muon_refusals(kw):
    assert muon(**kw) == 1


def test_muon_of_nothing():
    assert muon(rows=0) == muon(cols=0, w=None, g=None, m=None) == muon(count=0, ws=None, bytes=0) == 0
    assert muon(rows=0, lr=float("nan"), lr_dev=FAKE) == 0
    t = MuonTensors([], [], [])
    muon_step(t, lr=1e-3)
    with pytest.raises(_lib.MXError):
        muon_step(t, lr=1e-3, steps=0)


# ---- the Python entries


def test_orthogonalize_refusals():
    g = torch.zeros(8, 16)
    for bad in (lambda: orthogonalize(g[0]), lambda: orthogonalize(g.double()), lambda: orthogonalize(g.t()),
                lambda: orthogonalize(g, out=g), lambda: orthogonalize([g, g], out=[torch.zeros(8, 16)]),
                lambda: orthogonalize(g, out=torch.zeros(16, 8)), lambda: orthogonalize(g, out=torch.zeros(8, 16).half()),
                lambda: orthogonalize([g, g.double()]), lambda: orthogonalize(g.as_strided((4, 16), (8, 1)))):
        with pytest.raises(ValueError):
            bad()
    o = torch.zeros(8, 16)
    with pytest.raises(ValueError, match="share memory"):
        orthogonalize([g, g], out=[o, o])
    with pytest.raises(ValueError, match="share memory"):
        orthogonalize([g, o], out=[torch.zeros(8, 16), o[:8]])
    with pytest.raises(ValueError, match="CUDA"):
        orthogonalize([g, g], out=[o, torch.zeros(8, 16)])
    assert orthogonalize([]) == []


def test_the_list_of_a_step():
    w, g, m = torch.zeros(8, 16), torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(8, 16)
    h = torch.zeros(8, 16, dtype=torch.bfloat16)
    t = MuonTensors([w, w[:0]], [g, g[:0]], [m, m[:0]], copies=[h, None])
    assert (t._c[0].w, t._c[0].g, t._c[0].m, t._c[0].copy) == tuple(x.data_ptr() for x in (w, g, m, h))
    assert (t._c[0].rows, t._c[0].cols, t._c[0].grad, t._c[1].rows) == (8, 16, 1, 0)
    with pytest.raises(ValueError, match="CUDA"):
        muon_step(t, lr=1e-3)
    new = torch.zeros(8, 16)
    t.set_grads([new, new[:0]])
    assert (t._c[0].g, t._c[0].grad) == (new.data_ptr(), 0)
    for bad in ([new], [new, new], [new.double(), new[:0]], [new.t(), new[:0]], [w, new[:0]], [m, new[:0]]):
        with pytest.raises(ValueError):
            t.set_grads(bad)
    assert (t._c[0].g, t._c[0].grad) == (new.data_ptr(), 0)         # a refused call changes nothing
    for name in ("params", "grads", "momenta", "copies", "device"):
        with pytest.raises(AttributeError):
            setattr(t, name, [])
    for kw in (dict(adjust="none"), dict(grad_scale=2.0), dict(grad_scale=torch.zeros(2)), dict(lr=torch.zeros(2))):
        with pytest.raises(ValueError):
            muon_step(t, **(dict(lr=1e-3) | kw))


def test_lists_that_are_refused():
    w, g, m = torch.zeros(8, 16), torch.zeros(8, 16), torch.zeros(8, 16)
    buf = torch.zeros(300)
    for args in (([w], [g], []), ([w], [], [m]), ([w[0]], [g[0]], [m[0]]), ([w.bfloat16()], [g], [m]), ([w], [g], [w]),
                 ([w], [g], [m[:4]]), ([w.t()], [g.t()], [m.t()]), ([w, w], [g, g], [m, m.clone()]),
                 ([w], [g], [m], [m]), ([w], [g], [m], [g]), ([buf[:128].view(8, 16)], [g], [buf[127:255].view(8, 16)])):
        with pytest.raises(ValueError):
            MuonTensors(*args)
    MuonTensors([buf[:128].view(8, 16)], [g], [buf[128:256].view(8, 16)])
    MuonTensors([w, m], [g, g], [buf[:128].view(8, 16), buf[128:256].view(8, 16)])       # gradients may be shared


def test_structs_match_the_header():
    assert ctypes.sizeof(_lib.OrthoMatrixC) == 56 and ctypes.sizeof(_lib.OrthoParamsC) == 40
    assert ctypes.sizeof(_lib.MuonTensorC) == 56 and ctypes.sizeof(_lib.MuonParamsC) == 88


# ---- the documented error, on the oracle's model of the kernels' roundings


def model_error(g, **kw):
    ref = ortho.orthogonalize_ref(g, kw.get("steps", 5), kw.get("coefficients", ortho.COEFFICIENTS))
    return np.linalg.norm(ortho.orthogonalize_model(g, **kw) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("joined", [False, True])
def test_error_of_independent_roundings(joined):
    rng = np.random.default_rng(3)
    for m, n in ((64, 64), (96, 300), (130, 700)):
        low = rng.standard_normal((m, 4)) @ rng.standard_normal((4, n))
        for g in (rng.standard_normal((m, n)), rng.standard_t(2, (m, n)), weight_gradient(rng, m, n, 16), low,
                  rng.standard_normal((m, 1)) @ rng.standard_normal((1, n))):
            assert model_error(g, joined=joined) <= 2.6e-3
            assert model_error(g, joined=joined, steps=8) <= 4.5e-3
            assert model_error(g, joined=joined, coefficients=(2.0, -1.5, 0.5)) <= 1e-3
        assert model_error(low, joined=joined, steps=10) <= 5e-2


@pytest.mark.parametrize("joined", [False, True])
def test_error_of_roundings_that_are_alike(joined):
    """Constant matrices, in the model's own arithmetic on their one singular value: an entry e of a square of side m is
    the singular value m e.  The worst of many sizes stays within what is documented, and is no empty bound."""
    a, b, c = ortho.COEFFICIENTS
    half, sx, sa = ortho._half, ortho.SX, ortho.SA
    rng = np.random.default_rng(4)
    m = np.exp(rng.uniform(0, np.log(20000), 20000)).astype(int).astype(float)
    n = np.floor(m * np.exp(rng.uniform(0, 5, m.size)))

    def run(m, n):
        x = 1.0 / np.sqrt(m * n)
        hi = half(x, sx)
        low = half(x - hi, sx)
        if joined:
            s = half(hi * hi * n, sa)
            f0 = half(b * s + c * s * s * m, 1.0)
            p = half(a * s + f0 * s * m, sa)
            s = half(a * p + f0 * p * m, sa)
            f1 = half(b * s + c * s * s * m, 1.0)
            x = a * a * (hi + low) + half(a * f0 + a * f1 + f1 * f0 * m, 1.0) * m * hi
            hi = half(x, sx)
            low = half(x - hi, sx)
        for k in range(2 if joined else 0, 5):
            s = half(hi * hi * n, sa)
            f = b * s + c * s * s * m
            if k == 4:
                return (half(f, 1.0) * (m - 1) + half(f + a, 1.0)) * hi
            x = a * (hi + low) + half(f, 1.0) * m * hi
            hi = half(x, sx)
            low = half(x - hi, sx)

    # the short form is the model
    for p, q in ((40, 100), (85, 271)):
        whole = ortho.orthogonalize_model(np.ones((p, q)), eps=0.0, joined=joined)
        assert np.allclose(whole, run(float(p), float(q)), rtol=1e-12, atol=0)
    s = 1.0
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    off = np.abs(run(m, n) * np.sqrt(m * n) / s - 1)
    most = 2.5e-2 if joined else 1.5e-2
    assert 0.6 * most < off.max() <= most


def test_a_list_of_no_matrices_is_checked_as_any():
    assert orthogonalize([], out=[]) == []
    with pytest.raises(ValueError, match="1 outputs for 0 matrices"):
        orthogonalize([], out=[torch.zeros(8, 16)])
    for kw in (dict(steps=0), dict(eps=0.0), dict(coefficients=(5.0, 0.0, 0.0))):
        with pytest.raises(_lib.MXError):
            orthogonalize([], **kw)
