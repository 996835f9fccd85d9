"""CPU reference of the Newton-Schulz orthogonalization and of the Muon step, in float64 (test infrastructure).

orthogonalize_ref is the definition; orthogonalize_model rounds where the kernels round (float16 operands, X in two
parts), with exact sums in between, and so says what that rounding costs on a given matrix.
"""
import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
SX, SA = 4096.0, 2048.0


def orthogonalize_ref(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def _half(v, scale):
    return (v * scale).astype(np.float16).astype(np.float64) / scale


def orthogonalize_model(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7, joined=False):
    """joined: the first two steps as one (steps >= 3), as the kernels take them for lists of large, wide matrices."""
    a, b, c = coefficients
    x = np.asarray(g, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    hi = _half(x, SX)
    low = _half(x - hi, SX)
    first = 0
    if joined:
        s = _half(hi @ hi.T, SA)
        f0 = _half(b * s + c * (s @ s), 1.0)
        p = _half(a * s + f0 @ s, SA)
        s = _half(a * p + f0 @ p, SA)
        f1 = _half(b * s + c * (s @ s), 1.0)
        x = a * a * (hi + low) + _half(a * f0 + a * f1 + f1 @ f0, 1.0) @ hi
        hi = _half(x, SX)
        low = _half(x - hi, SX)
        first = 2
    for k in range(first, steps):
        s = _half(hi @ hi.T, SA)
        f = b * s + c * (s @ s)
        if k + 1 == steps:
            x = _half(f + a * np.eye(len(f)), 1.0) @ hi
        else:
            x = a * (hi + low) + _half(f, 1.0) @ hi
            hi = _half(x, SX)
            low = _half(x - hi, SX)
    return x.T if tall else x


def adjust_of(shape, adjust):
    rows, cols = shape
    return {"plain": 1.0, "rms": 0.2 * max(rows, cols) ** 0.5, "shape": max(1.0, rows / cols) ** 0.5}[adjust]


def muon_ref(w, g, m, lr, momentum=0.95, weight_decay=0.1, nesterov=True, steps=5, adjust="rms", eps=1e-7, scale=1.0):
    """(w, m, o) after one step, o the orthogonalized update."""
    w, m, g = (np.asarray(v, np.float64) for v in (w, m, g))
    g = g * scale
    m = m * momentum + g * (1.0 - momentum)
    o = orthogonalize_ref(g * (1.0 - momentum) + m * momentum if nesterov else m, steps, eps=eps)
    return w * (1.0 - lr * weight_decay) - o * (lr * adjust_of(w.shape, adjust)), m, o
