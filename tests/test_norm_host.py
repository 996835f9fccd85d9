"""Layer norm and its backward pass without a GPU: the oracle against closed forms and differences, and every refusal."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import _lib, layer_norm, layer_norm_grad
from oracle import norm

FAKE = 0x10000          # an aligned non-null address; validation never dereferences it


def test_forward_by_hand():
    x = np.array([[1.0, 3.0], [2.0, 2.0]])
    y, mean, rstd = norm.forward_ref(x, [2.0, 1.0], [0.5, 0.0], eps=1.0)
    assert mean.tolist() == [2.0, 2.0]
    assert np.allclose(rstd, [2 ** -0.5, 1.0], rtol=1e-15)
    assert np.allclose(y, [[0.5 - 2 * 2 ** -0.5, 2 ** -0.5], [0.5, 0.0]], rtol=1e-15)
    y, mean, rstd = norm.forward_ref(np.array([[3.0, 4.0]]), eps=0.0, kind="rms")
    assert np.allclose(y, [[3 / 12.5 ** 0.5, 4 / 12.5 ** 0.5]], rtol=1e-15)


def test_forward_against_torch():
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((5, 37)) + 3.0, rng.standard_normal(37), rng.standard_normal(37)
    want = torch.nn.functional.layer_norm(*(torch.from_numpy(v) for v in (x,)), (37,), torch.from_numpy(w),
                                          torch.from_numpy(b), 1e-5).numpy()
    assert np.allclose(norm.forward_ref(x, w, b)[0], want, rtol=1e-12, atol=1e-12)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (37,), torch.from_numpy(w), 1e-5).numpy()
    assert np.allclose(norm.forward_ref(x, w, kind="rms")[0], want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_against_differences(kind):
    """Central differences of sum(dy y) with step h in float64: off by about h^2 of the third derivative and 2^-53 / h."""
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((3, 11)) + 0.5, rng.standard_normal((3, 11))
    w, b = rng.standard_normal(11), rng.standard_normal(11) if kind == "layer" else None

    def loss(x, w, b):
        return float((dy * norm.forward_ref(x, w, b, 1e-2, kind)[0]).sum())

    _, mean, rstd = norm.forward_ref(x, w, b, 1e-2, kind)
    dx, dw, db = norm.backward_ref(dy, x, mean, rstd, w, kind)
    h = 1e-5
    for which, grad in ((0, dx), (1, dw)) + (((2, db),) if b is not None else ()):
        for at in np.ndindex(grad.shape):
            got = []
            for sign in (1, -1):
                args = [x.copy(), w.copy(), None if b is None else b.copy()]
                args[which][at] += sign * h
                got.append(loss(*args))
            assert abs((got[0] - got[1]) / (2 * h) - grad[at]) < 1e-7


# ---- refusals of the C entries


def fwd(x=FAKE, type=1, rows=4, cols=64, ld=64, w=FAKE, b=FAKE, wtype=1, eps=1e-5, kind=0, y=FAKE, ld_y=64, mean=FAKE,
        rstd=FAKE):
    return _lib.lib().mx_layer_norm(x, type, rows, cols, ld, w, b, wtype, eps, kind, y, ld_y, mean, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(rows=1 << 40), 1), (dict(cols=1 << 30), 1), (dict(type=2), 1),
    (dict(type=-1), 1), (dict(wtype=2), 1), (dict(kind=2), 1), (dict(kind=-1), 1), (dict(eps=-1e-9), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(eps=1e39), 1), (dict(x=None), 1),
    (dict(x=FAKE + 1), 1), (dict(x=FAKE + 2, type=0), 1), (dict(y=None), 1), (dict(y=FAKE + 1), 1), (dict(ld=63), 1),
    (dict(ld_y=63), 1), (dict(w=FAKE + 1), 1), (dict(w=FAKE + 2, wtype=0), 1), (dict(b=FAKE + 1), 1),
    (dict(mean=FAKE + 2), 1), (dict(rstd=FAKE + 2), 1), (dict(kind=1), 1), (dict(kind=1, b=None), 1),
    (dict(kind=1, mean=None), 1), (dict(rows=0), 0), (dict(cols=0), 0), (dict(rows=0, x=None, y=None), 0),
])
def test_forward_refusals(kw, want):
    assert fwd(**kw) == want


def bwd(dy=FAKE, ld_dy=64, x=FAKE, ld=64, type=1, rows=4, cols=64, w=FAKE, wtype=1, mean=FAKE, rstd=FAKE, kind=0, dx=FAKE,
        ld_dx=64, dw=FAKE, db=FAKE, ws=FAKE, bytes=1 << 30):
    return _lib.lib().mx_layer_norm_grad(dy, ld_dy, x, ld, type, rows, cols, w, wtype, mean, rstd, kind, dx, ld_dx, dw, db,
                                         ws, bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(rows=1 << 40), 1), (dict(cols=1 << 30), 1), (dict(type=2), 1),
    (dict(wtype=3), 1), (dict(kind=2), 1), (dict(dy=None), 1), (dict(dy=FAKE + 1), 1), (dict(x=None), 1),
    (dict(x=FAKE + 2, type=0), 1), (dict(dx=None), 1), (dict(dx=FAKE + 1), 1), (dict(ld=63), 1), (dict(ld_dy=63), 1),
    (dict(ld_dx=63), 1), (dict(w=FAKE + 1), 1), (dict(mean=None), 1), (dict(mean=FAKE + 2), 1), (dict(rstd=None), 1),
    (dict(rstd=FAKE + 2), 1), (dict(kind=1), 1), (dict(dw=FAKE + 2), 1), (dict(db=FAKE + 2), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 8), 1), (dict(bytes=100), 1), (dict(cols=0), 0),
])
def test_backward_refusals(kw, want):
    assert bwd(**kw) == want


def test_workspace_sizes():
    ask = _lib.lib().mx_layer_norm_grad_workspace
    for rows in (1, 33, 5000):
        for cols in (1, 64, 4096, 16384, 16385, 100000):
            need = ask(rows, cols, 1, 1)
            assert 8 * cols <= need <= 8 * 256 * cols + 8 * rows
            assert bwd(rows=rows, cols=cols, ld=cols, ld_dy=cols, ld_dx=cols, bytes=need - 1) == 1
    # dx alone: nothing but for rows too wide for a workgroup, whose two sums are kept
    assert ask(100, 4096, 1, 0) == 0 and ask(100, 100000, 1, 0) == 800
    for rows, cols, type in ((0, 5, 1), (5, 0, 1), (-1, 5, 1), (5, 1 << 30, 1), (1 << 62, 5, 0), (5, 5, 2)):
        assert ask(rows, cols, type, 1) == 0


# ---- refusals of the Python entries


def test_python_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    m, r = torch.zeros(4), torch.ones(4)
    for call in (lambda: layer_norm(x[0]), lambda: layer_norm(x.half()), lambda: layer_norm(x.t()),
                 lambda: layer_norm(x.as_strided((4, 64), (32, 1))), lambda: layer_norm(x, kind="batch"),
                 lambda: layer_norm(x, w[:63]), lambda: layer_norm(x, w.double()), lambda: layer_norm(x, w, w.bfloat16()),
                 lambda: layer_norm(x, w, w, kind="rms"), lambda: layer_norm(x, torch.ones(128)[::2]),
                 lambda: layer_norm(x, out=x[:2]), lambda: layer_norm(x, out=x.float()), lambda: layer_norm(x, out=x),
                 lambda: layer_norm_grad(x[:3], x, m, r), lambda: layer_norm_grad(x.float(), x, m, r),
                 lambda: layer_norm_grad(x, x, None, r), lambda: layer_norm_grad(x, x, m, r, kind="rms"),
                 lambda: layer_norm_grad(x, x, m[:3], r), lambda: layer_norm_grad(x, x, m, r.double()),
                 lambda: layer_norm_grad(x, x, m, r, w[:5]), lambda: layer_norm_grad(x, x, m, r, out=x),
                 lambda: layer_norm_grad(x, x, m, r, kind="other")):
        with pytest.raises(ValueError):
            call()
    # good arguments on the host reach the last check
    for call in (lambda: layer_norm(x, w), lambda: layer_norm_grad(x, x, m, r, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    buf = torch.zeros(4, 128, dtype=torch.bfloat16)
    for out, meets in ((buf[:, 64:], False), (buf[:, 63:127], True)):
        with pytest.raises(ValueError, match="share memory" if meets else "CUDA"):
            layer_norm(buf[:, :64], out=out)
