"""8-bit operands with a float32 scale for each block of 128, and their product (oracle side).

Test infrastructure only: see the package docstring.

A block is 128 consecutive values of a line ("line") or 128 lines x 128 values ("tile"); the last blocks of an axis
may be part-filled.  s = max(RN32(amax * RN32(1 / F)), 2^-126), r = RN32(1 / s), y = RN32(x * r), and the code is y
rounded to nearest, ties to the even code, in E4M3 (finite, largest 448) or E5M2 (largest finite 57344).  A block
holding Inf or NaN has s = NaN and codes 0.

The rounding is a nearest-level search over the table of all finite magnitudes, built from the bit fields.
"""
import numpy as np

FORMATS = {"e4m3": (4, 3, 7, 0x7E), "e5m2": (5, 2, 15, 0x7B)}     # exponent, mantissa bits, bias, largest finite code
BLOCK = 128


def levels(fmt):
    """The magnitudes of codes 0 .. largest finite, float64."""
    _, mbits, bias, top = FORMATS[fmt]
    code = np.arange(top + 1)
    e, m = code >> mbits, code & ((1 << mbits) - 1)
    return np.where(e == 0, m * 2.0 ** (1 - bias - mbits), (1 + m / (1 << mbits)) * 2.0 ** (e - bias))


def nearest_code(mag, table):
    """The code whose level is nearest to each magnitude (float64), ties to the even code, saturating."""
    hi = np.clip(np.searchsorted(table, mag), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = mag - table[lo], table[hi] - mag
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def decode(codes, fmt):
    table = levels(fmt)
    mag = np.append(table, np.full(128 - len(table), np.nan))[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag)


def bf16_values(bits):
    return (np.asarray(bits).view(np.uint16).astype(np.uint32) << 16).view(np.float32)


def scales_of(amax, largest):
    """s and r = RN32(1 / s) of each block's float32 amax (NaN or Inf: s = NaN, r = 0)."""
    with np.errstate(all="ignore"):
        s = np.maximum(amax * (np.float32(1) / np.float32(largest)), np.float32(2.0 ** -126)).astype(np.float32)
        r = (np.float32(1.0) / s).astype(np.float32)
    bad = ~np.isfinite(amax)
    return np.where(bad, np.float32(np.nan), s), np.where(bad, np.float32(0), r)


def quantize_lines(x, kind, fmt):
    """(codes (L, padded K), scales) of float32 lines x."""
    lines, k = x.shape
    kb, lb = -(-k // BLOCK), -(-lines // BLOCK)
    v = np.zeros((lb * BLOCK, kb * BLOCK), dtype=np.float32)
    v[:lines, :k] = x
    mag = np.where(np.isnan(v), np.float32(np.inf), np.abs(v))
    table = levels(fmt)
    if kind == "line":
        s, r = scales_of(mag.reshape(-1, kb, BLOCK).max(axis=2), table[-1])
        each, scales = np.repeat(r, BLOCK, axis=1), np.ascontiguousarray(s[:lines].T)
    else:
        s, r = scales_of(mag.reshape(lb, BLOCK, kb, BLOCK).max(axis=(1, 3)), table[-1])
        each, scales = np.repeat(np.repeat(r, BLOCK, axis=0), BLOCK, axis=1), s
    with np.errstate(invalid="ignore"):
        y = (v * each).astype(np.float32)
    y = np.where(each == 0, np.float32(0), y)
    code = nearest_code(np.abs(y).astype(np.float64), table) | np.where(np.signbit(y), 0x80, 0)
    return np.where(each == 0, 0, code).astype(np.uint8)[:lines], scales


def quantize_ref(bits, axis, kind, fmt):
    """{"row": (codes, scales), "col": (codes, scales)} of a bf16 matrix given by its bit patterns."""
    x = bf16_values(bits)
    out = {}
    if axis != "col":
        out["row"] = quantize_lines(x, kind, fmt)
    if axis != "row":
        out["col"] = quantize_lines(np.ascontiguousarray(x.T), kind, fmt)
    return out


def values(codes, scales, kind, fmt):
    """float64 values (L, padded K) of an operand."""
    lines = codes.shape[0]
    s = scales.T if kind == "line" else np.repeat(scales, BLOCK, axis=0)[:lines]
    return decode(codes, fmt) * np.repeat(s.astype(np.float64), BLOCK, axis=1)


def gemm_ref(a, a_fmt, b, b_fmt, b_kind):
    """(C, G): the float64 product of two (codes, scales) operands and sum_k |a b|."""
    av, bv = values(*a, "line", a_fmt), values(*b, b_kind, b_fmt)
    return av @ bv.T, np.abs(av) @ np.abs(bv).T
