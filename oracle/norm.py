"""CPU reference of layer norm, its RMS form and their backward pass, in float64 (test infrastructure)."""
import numpy as np


def forward_ref(x, weight=None, bias=None, eps=1e-5, kind="layer"):
    """(y, mean, rstd) of the rows of x; mean is zero for kind "rms"."""
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    mean = x.sum(axis=1) / n if kind == "layer" else np.zeros(x.shape[0])
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / n + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def backward_ref(dy, x, mean, rstd, weight=None, kind="layer"):
    """(dx, dweight, dbias) for the statistics given."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    n = x.shape[1]
    h = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    inner = g - h * ((g * h).sum(axis=1) / n)[:, None]
    if kind == "layer":
        inner = inner - (g.sum(axis=1) / n)[:, None]
    return inner * np.asarray(rstd, np.float64)[:, None], (dy * h).sum(axis=0), dy.sum(axis=0)
