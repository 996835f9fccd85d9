"""One AdamW step on float32 weights with 32-bit or 8-bit moments (oracle side).

Test infrastructure only: see the package docstring.

Decoupled weight decay, float32 with one rounding per operation in the order written; the coefficients come from
float64.  8-bit moments have a float32 scale for each 128 elements of the flattened tensor: the first in E4M3, the
second in E5M3 (5 exponent bits, 3 mantissa bits, bias 15, no sign; codes up to 0xF7 = 61440).  A moment is
code * scale; after the step s = max(RN32(amax * RN32(1 / F)), 2^-126), F = 448 or 61440, and
y = RN32(value * RN32(1 / s)) goes to the nearest level, ties to the even code, or up from the level below iff
floor(f 2^16) + r >= 2^16 with f the fraction of the step and r the element's 16-bit draw.  A second moment above 0
keeps at least code 1; a block holding Inf or NaN gets s = NaN and codes 0.
"""
import numpy as np

from .fp8 import BLOCK, levels, nearest_code, scales_of
from .philox import uniform_halfwords

E4M3 = levels("e4m3")


def e5m3_levels():
    code = np.arange(0xF8)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -17, (8 + m) * 2.0 ** (e - 18.0))


E5M3 = e5m3_levels()


def coefficients(lr, beta1, beta2, eps, weight_decay, step):
    f = np.float32
    return {"b1": f(beta1), "n1": f(1.0 - beta1), "b2": f(beta2), "n2": f(1.0 - beta2), "eps": f(eps),
            "c1": f(lr / (1.0 - beta1 ** step)), "c2": f(1.0 / np.sqrt(1.0 - beta2 ** step)),
            "keep": f(1.0 - lr * weight_decay)}


def update(w, g, m, v, c, grad_scale=None):
    """(w, m, v) after the step, float32."""
    with np.errstate(all="ignore"):
        if grad_scale is not None:
            g = g * np.float32(grad_scale)
        m = m * c["b1"] + g * c["n1"]
        v = v * c["b2"] + g * c["n2"] * g
        d = np.sqrt(v) * c["c2"] + c["eps"]
        w = w * c["keep"] - m / d * c["c1"]
    for x in (w, m, v):
        assert x.dtype == np.float32
    return w, m, v


def decode_state(codes, scales, first):
    table = np.append(E4M3, np.nan) if first else np.append(E5M3, [np.nan] * 8)
    mag = table[codes & 0x7F if first else codes].astype(np.float32)
    val = np.where(codes & 0x80, -mag, mag) if first else mag
    return (val * np.repeat(scales, BLOCK)[:len(codes)]).astype(np.float32)


def encode_state(x, first, seed=None, stream=None):
    """(codes, scales) of float32 moments; seed None: round to nearest."""
    n = len(x)
    v = np.zeros(-(-n // BLOCK) * BLOCK, dtype=np.float32)
    v[:n] = x
    table = E4M3 if first else E5M3
    s, r = scales_of(np.where(np.isnan(v), np.float32(np.inf), np.abs(v)).reshape(-1, BLOCK).max(axis=1), table[-1])
    each = np.repeat(r, BLOCK)[:n]
    with np.errstate(invalid="ignore"):
        y = np.where(each == 0, np.float32(0), x * each).astype(np.float32)
    mag = np.abs(y).astype(np.float64)
    if seed is None:
        code = nearest_code(mag, table)
    else:
        lo = np.clip(np.searchsorted(table, mag, side="right") - 1, 0, len(table) - 1)
        hi = np.minimum(lo + 1, len(table) - 1)
        gap = np.where(hi > lo, table[hi] - table[lo], 1.0)
        f = np.floor((mag - table[lo]) / gap * 65536.0)
        draw = uniform_halfwords(seed, stream, np.arange(n, dtype=np.uint64))
        code = np.where(f + draw >= 65536.0, hi, lo)
    if first:
        code = code | np.where(np.signbit(x), 0x80, 0)
    else:
        code = np.where(x > 0, np.maximum(code, 1), code)
    return np.where(each == 0, 0, code).astype(np.uint8), s


def step8(w, g, state, c, grad_scale=None, seed=None, ordinal=0):
    """(w, (m codes, m scales, v codes, v scales)) of one tensor after a step with 8-bit moments."""
    mc, ms, vc, vs = state
    w, m, v = update(w, g, decode_state(mc, ms, True), decode_state(vc, vs, False), c, grad_scale)
    return w, encode_state(m, True, seed, 4 + 2 * ordinal) + encode_state(v, False, seed, 5 + 2 * ordinal)
