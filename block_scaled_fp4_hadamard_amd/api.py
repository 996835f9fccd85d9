"""PyTorch-facing wrappers over the C ABI: they allocate outputs with torch on
the tensor's device and launch on torch's current stream.  No arithmetic of
the method happens here.
"""
from bisect import bisect_left
from dataclasses import dataclass

import torch

from . import _lib

GEMM_GROUP_MAX = _lib.GEMM_GROUP_MAX    # problems per gemm_grouped call


@dataclass
class QTensor:
    """A block-scaled 4-bit operand: L lines of length K, K-contiguous.

    codes  uint8 (L, K/2): element 2j of a line in the low nibble of byte j
    scales uint8 (L, K/block): E8M0 exponent byte per block of `block` (32, or 16) elements
    """
    codes: torch.Tensor
    scales: torch.Tensor
    grid: str = "e2m1"
    block: int = 32           # values per E8M0 scale: scales hold K / block bytes per line

    @property
    def lines(self):
        return self.codes.shape[0]

    @property
    def k(self):
        return self.codes.shape[1] * 2

    def c_struct(self):
        return _lib.qtensor(self.codes.data_ptr(), self.codes.stride(0),
                            self.scales.data_ptr(), self.scales.stride(0))


def _stream(dev):
    if dev.type != "cuda":
        return None       # host tensors reach only the library's argument checks, which launch nothing
    return ctypes_void(torch.cuda.current_stream(dev).cuda_stream)


def ctypes_void(handle):
    return handle if handle else None


def _bits_view(x):
    if x.dtype == torch.bfloat16:
        return x.view(torch.int16)
    if x.dtype in (torch.int16, torch.uint16):
        return x
    raise TypeError("x must be bfloat16 (or its 16-bit patterns), got %s" % x.dtype)


def empty_qtensor(lines, k, device, grid="e2m1", block=32):
    """An output operand; scale rows are padded to a multiple of 4 bytes, which the GEMM's copy path needs
    (the padding is never read as data)."""
    nb = k // block
    scales = torch.empty((lines, (nb + 3) // 4 * 4), dtype=torch.uint8, device=device)[:, :nb]
    return QTensor(torch.empty((lines, k // 2), dtype=torch.uint8, device=device), scales, grid, block)


def quantize(x, axis="row", grid="e2m1", rounding="rtne", seed=0, had_n=0, had_kind="det", had_seed=0,
             block=32, row_out=None, col_out=None):
    """Quantize a 2-D bf16 CUDA tensor; returns {"row": QTensor, "col": QTensor} as requested.

    had_n 0 means no rotation; otherwise 16 or 32 with had_kind "det" or "rand".
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    xb = _bits_view(x)
    rows, cols = x.shape
    dev = x.device
    do_row, do_col = axis in ("row", "both"), axis in ("col", "both")
    for given in (row_out, col_out):
        if given is not None and given.block != block:
            raise ValueError("an output operand of block %d given for block %d" % (given.block, block))
    out = {}
    rq = cq = None
    if do_row:
        out["row"] = row_out if row_out is not None else empty_qtensor(rows, cols, dev, grid, block)
        rq = out["row"].c_struct()
    if do_col:
        out["col"] = col_out if col_out is not None else empty_qtensor(cols, rows, dev, grid, block)
        cq = out["col"].c_struct()
    stream = _stream(dev)
    if had_n:
        st = _lib.mx_hadamard_quantize(xb.data_ptr(), rows, cols, xb.stride(0), block, _lib.GRID[grid],
                                       _lib.ROUND[rounding], _lib.AXIS[axis], seed, had_n, _lib.HAD[had_kind],
                                       had_seed, rq, cq, stream)
        _lib.check(st, "mx_hadamard_quantize")
    else:
        st = _lib.mx_quantize(xb.data_ptr(), rows, cols, xb.stride(0), block, _lib.GRID[grid],
                              _lib.ROUND[rounding], _lib.AXIS[axis], seed, rq, cq, stream)
        _lib.check(st, "mx_quantize")
    return out


def gemm(a, b, out_dtype=torch.float32, out=None, grid=None):
    """C = A B^T on the decoded operands (M x N), fp32 accumulation, fp32 or bf16 output.

    The operands' block size goes to the library as it is (a 16-value operand is refused there: the matrix
    cores take 32-value blocks).
    """
    if a.k != b.k:
        raise ValueError("operands disagree on K: %d vs %d" % (a.k, b.k))
    if a.block != b.block:
        raise ValueError("operands disagree on the block size: %d vs %d" % (a.block, b.block))
    for name, q in (("a", a), ("b", b)):
        if q.scales.shape[1] * q.block != q.k:
            raise ValueError("%s: %d scale bytes per line do not cover K = %d in blocks of %d"
                             % (name, q.scales.shape[1], q.k, q.block))
    grid = grid or a.grid
    M, N, K = a.lines, b.lines, a.k
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.codes.device)
    elif out.dim() != 2 or out.shape[0] != M or out.shape[1] != N or out.stride(1) != 1:
        raise ValueError("out must be a row-major (%d, %d) view" % (M, N))
    kind = {torch.float32: "f32", torch.bfloat16: "bf16"}[out.dtype]
    st = _lib.mx_gemm(a.c_struct(), b.c_struct(), M, N, K, _lib.GRID[grid], a.block, out.data_ptr(), out.stride(0),
                      _lib.OUT[kind], _stream(out.device))
    _lib.check(st, "mx_gemm")
    return out


def gemm_grouped(problems, grid=None):
    """Several GEMMs C_i = A_i B_i^T of one K, grid and output dtype in one library call.

    problems: list of (a, b, out) with out a preallocated (M_i, N_i) fp32 or bf16 tensor.  Each result is
    the one gemm(a, b, out=out) gives, to the bit; the library runs them as one launch when they can share
    it and one launch each otherwise.
    """
    if not problems:
        return []
    if len(problems) > GEMM_GROUP_MAX:
        raise ValueError("at most %d problems per call" % GEMM_GROUP_MAX)
    a0, _, out0 = problems[0]
    grid = grid or a0.grid
    kinds = {torch.float32: "f32", torch.bfloat16: "bf16"}
    args = []
    for i, (a, b, out) in enumerate(problems):
        if a.k != a0.k or b.k != a0.k:
            raise ValueError("problem %d: every operand must have K = %d" % (i, a0.k))
        if a.block != a0.block or b.block != a0.block:
            raise ValueError("problem %d: operands disagree on the block size" % i)
        if out.dtype != out0.dtype:
            raise ValueError("problem %d: every output must be %s" % (i, out0.dtype))
        if out.dim() != 2 or out.shape[0] != a.lines or out.shape[1] != b.lines or out.stride(1) != 1:
            raise ValueError("problem %d: out must be a row-major (%d, %d) view" % (i, a.lines, b.lines))
        for name, q in (("a", a), ("b", b)):
            if q.scales.shape[1] * q.block != q.k:
                raise ValueError("problem %d, %s: %d scale bytes per line do not cover K = %d in blocks of %d"
                                 % (i, name, q.scales.shape[1], q.k, q.block))
        args.append((a.c_struct(), b.c_struct(), a.lines, b.lines, out.data_ptr(), out.stride(0)))
    st = _lib.mx_gemm_grouped(args, a0.k, _lib.GRID[grid], a0.block, _lib.OUT[kinds[out0.dtype]],
                              _stream(out0.device))
    _lib.check(st, "mx_gemm_grouped")
    return [out for _, _, out in problems]


def mxnorm_quantize(x, power, c, grid="e2m1", rounding="rtne", seed=0, out=None, rho=None):
    """MXNorm of every row of a 2-D bf16 CUDA tensor fused with its row-wise MX cast.

    Returns (QTensor of the normalized rows, rho float32 (rows,)).  c is the caller's correction constant
    c(power, 32) (precomputed once on the host, e.g. by mxnorm_constant.correction).
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    xb = _bits_view(x)
    rows, cols = x.shape
    dev = x.device
    c = float(c)
    q = out if out is not None else empty_qtensor(rows, cols, dev, grid)
    r = rho if rho is not None else torch.empty((rows,), dtype=torch.float32, device=dev)
    st = _lib.mx_mxnorm_quantize(xb.data_ptr(), rows, cols, xb.stride(0), power, c, _lib.GRID[grid],
                                 _lib.ROUND[rounding], seed, q.c_struct(), r.data_ptr(), _stream(dev))
    _lib.check(st, "mx_mxnorm_quantize")
    return q, r


def quant_stats(x, q, axis="row", grid=None, had_n=0, had_kind="det", had_seed=0, stats=None, to_host=True):
    """Diagnostic totals of one quantized output q of x, as the kernel accumulates them: sum of y^2, sum of
    (y - y_hat)^2, the counts of the 8 magnitude codes and the number of blocks.  stats: an optional zeroed
    float64 (12,) CUDA tensor to reuse.  Ratios built from these (SQNR, bucket usage) are the caller's.
    to_host=False returns the stats tensor itself, with no copy to the host and no synchronization (the
    kernel adds to it: zero it before a call whose totals are read).
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    xb = _bits_view(x)
    rows, cols = x.shape
    grid = grid or q.grid
    buf = stats if stats is not None else torch.zeros(12, dtype=torch.float64, device=x.device)
    st = _lib.mx_quant_stats(xb.data_ptr(), rows, cols, xb.stride(0), _lib.AXIS[axis], _lib.GRID[grid],
                             had_n, _lib.HAD["none" if not had_n else had_kind], had_seed, q.c_struct(),
                             buf.data_ptr(), _stream(x.device))
    _lib.check(st, "mx_quant_stats")
    if not to_host:
        return buf
    host = buf.cpu()
    counts = host[2:].view(torch.int64)
    return {"sum_sq": float(host[0]), "sum_err_sq": float(host[1]), "hist": [int(v) for v in counts[:8]],
            "blocks": int(counts[8])}


def hadamard_rotate(x, axis="row", had_n=32, had_kind="det", had_seed=0, out=None):
    """The block Hadamard rotation alone: a float32 CUDA tensor, (rows, cols) for axis "row" (rotated along
    rows), or the transpose (cols, rows) for axis "col" (rotated along columns)."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    xb = _bits_view(x)
    rows, cols = x.shape
    shape = (rows, cols) if axis == "row" else (cols, rows)
    y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=x.device)
    if tuple(y.shape) != shape or y.dtype != torch.float32 or y.stride(1) != 1:
        raise ValueError("out must be a float32 %s tensor with unit column stride" % (shape,))
    st = _lib.mx_hadamard_rotate(xb.data_ptr(), rows, cols, xb.stride(0), had_n, _lib.HAD[had_kind], had_seed,
                                 _lib.AXIS[axis], y.data_ptr(), y.stride(0), _stream(x.device))
    _lib.check(st, "mx_hadamard_rotate")
    return y


def quantize_f32(y, axis="row", grid="e2m1", rounding="rtne", seed=0, out=None):
    """The MX cast of the lines of a float32 CUDA tensor y (lines, len); axis names which output of the original
    tensor the lines are ("col": y holds its transpose), which selects the stochastic-rounding stream."""
    if y.dim() != 2 or y.stride(1) != 1 or y.dtype != torch.float32:
        raise ValueError("y must be a 2-D float32 tensor with unit column stride")
    lines, length = y.shape
    q = out if out is not None else empty_qtensor(lines, length, y.device, grid)
    st = _lib.mx_quantize_f32(y.data_ptr(), lines, length, y.stride(0), _lib.GRID[grid], _lib.ROUND[rounding],
                              _lib.AXIS[axis], seed, q.c_struct(), _stream(y.device))
    _lib.check(st, "mx_quantize_f32")
    return q


@dataclass
class OsciState:
    """OsciReset's per-element state, float32 tensors shaped like the master weights."""
    w_prev: torch.Tensor
    q_prev: torch.Tensor
    dist_m: torch.Tensor
    dist_q: torch.Tensor

    @staticmethod
    def empty_like(w):
        return OsciState(*(torch.empty_like(w) for _ in range(4)))


def osci_reset(w, q, state, mode, threshold=0.0, resets=None):
    """One OsciReset step on float32 master weights w (rows, cols) given q, their row-wise quantization (a
    QTensor, block 32); mode "init", "track" or "check".  resets: an optional int64 CUDA tensor of one element
    to which the number of reset elements is added.  w is updated in place."""
    if w.dim() != 2 or w.stride(1) != 1 or w.dtype != torch.float32:
        raise ValueError("w must be a 2-D float32 tensor with unit column stride")
    for t in (state.q_prev, state.dist_m, state.dist_q):
        if t.stride() != state.w_prev.stride() or t.shape != w.shape:
            raise ValueError("the state tensors must share w's shape and one row stride")
    rows, cols = w.shape
    st = _lib.mx_osci_reset(w.data_ptr(), rows, cols, w.stride(0), q.c_struct(), _lib.GRID[q.grid],
                            state.w_prev.data_ptr(), state.q_prev.data_ptr(), state.dist_m.data_ptr(),
                            state.dist_q.data_ptr(), state.w_prev.stride(0), _lib.OSCI[mode], threshold,
                            resets.data_ptr() if resets is not None else None, _stream(w.device))
    _lib.check(st, "mx_osci_reset")
    return w


@dataclass
class NVTensor:
    """An NVFP4-style double-block operand: L lines of length K.

    codes uint8 (L, K/2) E2M1 as QTensor; inner uint8 (L, K/16) E4M3 scales; outer float32 (L, K/128)
    """
    codes: torch.Tensor
    inner: torch.Tensor
    outer: torch.Tensor

    def c_struct(self):
        return _lib.nvtensor(self.codes.data_ptr(), self.codes.stride(0), self.inner.data_ptr(),
                             self.inner.stride(0), self.outer.data_ptr(), self.outer.stride(0))


def nvfp4_quantize(x, axis="row", rounding="rtne", seed=0, row_out=None, col_out=None):
    """NVFP4-style double-block quantization of a 2-D bf16 CUDA tensor; {"row": NVTensor, "col": NVTensor}.

    row_out / col_out reuse NVTensors from an earlier call of the same shape.
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit column stride")
    xb = _bits_view(x)
    rows, cols = x.shape
    dev = x.device

    def empty(lines, k):
        return NVTensor(torch.empty((lines, k // 2), dtype=torch.uint8, device=dev),
                        torch.empty((lines, k // 16), dtype=torch.uint8, device=dev),
                        torch.empty((lines, k // 128), dtype=torch.float32, device=dev))
    out = {}
    if axis in ("row", "both"):
        out["row"] = row_out if row_out is not None else empty(rows, cols)
    if axis in ("col", "both"):
        out["col"] = col_out if col_out is not None else empty(cols, rows)
    rq = out["row"].c_struct() if "row" in out else None
    cq = out["col"].c_struct() if "col" in out else None
    st = _lib.mx_nvfp4_quantize(xb.data_ptr(), rows, cols, xb.stride(0), _lib.ROUND[rounding], _lib.AXIS[axis],
                                seed, rq, cq, _stream(dev))
    _lib.check(st, "mx_nvfp4_quantize")
    return out


FP8_BLOCK = 128           # values per scale (MX_FP8_BLOCK)


def _fp8_blocks(n):
    return -(-n // FP8_BLOCK)


# told which of the caller's tensors a kernel wrote, autograd refuses a backward that would read the old values
_written = torch.autograd.graph.increment_version
_FP8_FMT, _FP8_KIND, _Fp8TensorC = _lib.FP8_FMT, _lib.FP8_KIND, _lib.Fp8TensorC
_OUT_KINDS = {torch.float32: _lib.OUT["f32"], torch.bfloat16: _lib.OUT["bf16"]}


def _pitch(stride, rows, cols, name):
    """Elements between the rows of a rows x cols tensor of this stride, whose rows are whole and do not overlap."""
    ld, one = stride
    if cols > 1 and one != 1:
        raise ValueError("%s must have unit column stride" % name)
    if rows > 1 and ld < cols:
        raise ValueError("%s: its rows overlap (a stride of %d for %d columns)" % (name, ld, cols))
    return ld if rows > 1 else cols


def _meet(x, y):
    """Whether two regions of memory share a byte, each (address, rows, bytes of a row, bytes between rows)."""
    (p, rows_p, wide_p, pitch_p), (q, rows_q, wide_q, pitch_q) = x, y
    if p + (rows_p - 1) * pitch_p + wide_p <= q or q + (rows_q - 1) * pitch_q + wide_q <= p:
        return False
    if not (rows_p and wide_p and rows_q and wide_q):
        return False
    # each row of x against the last row of y that starts before its end: views side by side in one buffer are apart
    start = p + pitch_p * torch.arange(rows_p, device="cpu")
    other = q + pitch_q * torch.arange(rows_q, device="cpu")
    last = torch.searchsorted(other, start + wide_p) - 1
    return bool(((last >= 0) & (other[last.clamp_min(0)] + wide_q > start)).any())


def _launch(at, name, entry, *args):
    """entry(*args, stream) on the current stream of CUDA device number `at`, as the current device; a number below 0,
    a host tensor's, is refused."""
    if at < 0:
        raise ValueError("the operands must be CUDA tensors")
    stream = torch._C._cuda_getCurrentRawStream(at) or None
    if at == torch.cuda.current_device():
        st = entry(*args, stream)
    else:
        with torch.cuda.device(at):
            st = entry(*args, stream)
    if st:
        raise _lib.MXError(st, name)


@dataclass
class Fp8Tensor:
    """A block-scaled 8-bit operand: L lines of length k, K-contiguous.

    codes  uint8 (L, 128 * ceil(k / 128)): E4M3 or E5M2 bytes, zeros past k
    scales float32: kind "line" (ceil(k / 128), L), one per line and 128 values; kind "tile"
           (ceil(L / 128), ceil(k / 128)), one per 128 lines x 128 values
    """
    codes: torch.Tensor
    scales: torch.Tensor
    k: int
    fmt: str = "e4m3"
    kind: str = "line"

    @property
    def lines(self):
        return self.codes.shape[0]

    def check(self, name):
        """The operand as the library takes it; ValueError if its tensors are not what the class describes."""
        codes, scales, kind = self.codes, self.scales, self.kind
        if self.fmt not in _FP8_FMT or kind not in _FP8_KIND:
            raise ValueError("%s: unknown format %r or kind %r" % (name, self.fmt, kind))
        kb = -(-self.k // 128)
        shape = codes.shape
        if codes.dtype != torch.uint8 or len(shape) != 2 or shape[1] != kb * 128:
            raise ValueError("%s: codes must be uint8 (lines, %d) for k = %d" % (name, kb * 128, self.k))
        lines, width = shape
        rows, cols = (kb, lines) if kind == "line" else (-(-lines // 128), kb)
        if scales.dtype != torch.float32 or scales.shape != (rows, cols):
            raise ValueError("%s: scales must be float32 %s for kind %r" % (name, (rows, cols), kind))
        if scales.get_device() != codes.get_device():
            raise ValueError("%s: codes and scales are on different devices" % name)
        return _Fp8TensorC(codes.data_ptr(), _pitch(codes.stride(), lines, width, name),
                           scales.data_ptr(), _pitch(scales.stride(), rows, cols, name))

    def c_struct(self):
        return self.check("operand")


def empty_fp8(lines, k, device, fmt="e4m3", kind="line"):
    """An uninitialised output operand."""
    kb = _fp8_blocks(k)
    shape = (kb, lines) if kind == "line" else (_fp8_blocks(lines), kb)
    return Fp8Tensor(torch.empty((lines, kb * FP8_BLOCK), dtype=torch.uint8, device=device),
                     torch.empty(shape, dtype=torch.float32, device=device), k, fmt, kind)


def fp8_quantize(x, axis="row", kind="line", fmt="e4m3", row_out=None, col_out=None):
    """Cast a 2-D bf16 CUDA tensor to 8 bits with a float32 scale for each block of 128 (a line's 128 values, kind
    "line", or a 128 x 128 tile, "tile"); {"row": Fp8Tensor of x's rows, "col": of its columns} as requested.

    x needs a column count and a row stride that are multiples of 8.
    """
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError("x must be bfloat16 (or its 16-bit patterns), got %s" % x.dtype)
    if axis not in _lib.AXIS or kind not in _lib.FP8_KIND or fmt not in _lib.FP8_FMT:
        raise ValueError("unknown axis %r, kind %r or format %r" % (axis, kind, fmt))
    rows, cols = x.shape
    ld = _pitch(x.stride(), rows, cols, "x")
    dev = x.device
    out = {}
    c = [None, None]
    if axis != "col":
        q = row_out if row_out is not None else empty_fp8(rows, cols, dev, fmt, kind)
        out["row"], c[0] = q, _fp8_output(q, row_out is not None, "row_out", rows, cols, fmt, kind, dev)
    if axis != "row":
        q = col_out if col_out is not None else empty_fp8(cols, rows, dev, fmt, kind)
        out["col"], c[1] = q, _fp8_output(q, col_out is not None, "col_out", cols, rows, fmt, kind, dev)
    if row_out is not None or col_out is not None:
        given = [("x", (x.data_ptr(), rows, 2 * cols, 2 * ld))]
        for name, q, s in (("row_out", row_out, c[0]), ("col_out", col_out, c[1])):
            if q is None or s is None:
                continue
            for part in _regions(q, s):
                for other, region in given:
                    if _meet(part, region):
                        raise ValueError("%s and %s share memory" % (other, name))
                given.append((name, part))
    _launch(x.get_device(), "mx_fp8_quantize", _lib.lib().mx_fp8_quantize, x.data_ptr(), rows, cols, ld, _FP8_FMT[fmt],
            _FP8_KIND[kind], _lib.AXIS[axis], *c)
    for q, s in ((row_out, c[0]), (col_out, c[1])):
        if q is not None and s is not None:
            _written((q.codes, q.scales))
    return out


def _regions(q, c):
    """The memory of an operand's codes and of its scales, as _meet takes it."""
    lines, width = q.codes.shape
    rows, cols = q.scales.shape
    return (c.codes or 0, lines, width, c.ld_codes), (c.scales or 0, rows, 4 * cols, 4 * c.ld_scales)


def _fp8_output(q, given, name, lines, k, fmt, kind, dev):
    """An output operand as the library takes it: checked if it is the caller's, plain if it was made just now."""
    if not given:
        return _lib.Fp8TensorC(q.codes.data_ptr(), q.codes.shape[1], q.scales.data_ptr(), q.scales.shape[1])
    if (q.lines, q.k, q.fmt, q.kind) != (lines, k, fmt, kind) or q.codes.device != dev:
        raise ValueError("%s is not an %s operand of %d %s lines of %d values on %s" % (name, fmt, lines, kind, k, dev))
    return q.check(name)


def fp8_gemm(a, b, out_dtype=torch.float32, out=None):
    """C = A B^T (M x N) on two 8-bit operands' values, fp32 accumulation, fp32 or bf16 output.

    a is scaled by lines (kind "line"), b by lines or tiles; each may be E4M3 or E5M2.  bf16 output runs on the 8-bit
    matrix instruction; fp32 output on the bf16 one, whose products are exact, at half its rate.
    """
    ca, cb = a.check("a"), b.check("b")
    if a.k != b.k:
        raise ValueError("operands disagree on K: %d vs %d" % (a.k, b.k))
    if a.kind != "line":
        raise ValueError("a must be scaled by lines, got kind %r" % a.kind)
    at = a.codes.get_device()
    M, N = a.codes.shape[0], b.codes.shape[0]
    fresh = out is None
    if fresh:
        out = a.codes.new_empty((M, N), dtype=out_dtype)
    elif out.dim() != 2 or out.shape[0] != M or out.shape[1] != N:
        raise ValueError("out must be a row-major (%d, %d) view" % (M, N))
    kind = _OUT_KINDS.get(out.dtype)
    if kind is None:
        raise ValueError("the output must be float32 or bfloat16, got %s" % out.dtype)
    if b.codes.get_device() != at or out.get_device() != at:
        raise ValueError("a, b and out must be on one device")
    ldc = _pitch(out.stride(), M, N, "out")
    if not fresh:
        size = out.element_size()
        region = (out.data_ptr(), M, size * N, size * ldc)
        for name, q, c in (("a", a, ca), ("b", b, cb)):
            for part in _regions(q, c):
                if _meet(region, part):
                    raise ValueError("out and %s share memory" % name)
    lib = _lib.lib()
    # the workspace is this call's own: held until the launch, its memory then goes to later work of this stream only
    size = lib.mx_fp8_gemm_workspace(M, N, a.k, kind)
    space = a.codes.new_empty(size) if size else None
    _launch(at, "mx_fp8_gemm", lib.mx_fp8_gemm, ca, _FP8_FMT[a.fmt], cb, _FP8_FMT[b.fmt], _FP8_KIND[b.kind], M, N, a.k,
            out.data_ptr(), ldc, kind, space.data_ptr() if size else None, size)
    if not fresh:
        _written(out)
    return out


@dataclass
class AdamWState:
    """AdamW's moments of one tensor of n elements: float32 m and v, or (8 bits) uint8 E4M3 m and E5M3 v with float32
    scales for each 128 elements."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor = None
    v_scale: torch.Tensor = None

    @staticmethod
    def zeros_like(w, bits=32):
        """The state of a first step: all moments zero."""
        if bits == 32:
            return AdamWState(torch.zeros_like(w), torch.zeros_like(w))
        if bits != 8:
            raise ValueError("states are held in 8 or 32 bits, not %r" % (bits,))
        codes = [torch.zeros(w.shape, dtype=torch.uint8, device=w.device) for _ in range(2)]
        scales = [torch.zeros(_fp8_blocks(w.numel()), dtype=torch.float32, device=w.device) for _ in range(2)]
        return AdamWState(*codes, *scales)

    @property
    def bits(self):
        return 8 if self.m.dtype == torch.uint8 else 32


class AdamWTensors:
    """The tensors that adamw_step updates, checked and laid out once: float32 master weights, their gradients
    (float32 or bf16), their states (all of 8 or all of 32 bits) and, if given, the bf16 copies that a step writes.

    Every tensor is contiguous, and none that a step writes may share memory with another or with a gradient.  The
    object holds the tensors it was given: params, grads, states and copies are read-only, a state's field replaced
    later is not seen, and a tensor whose storage is replaced (Tensor.data, resize_) needs a new object.  New gradient
    tensors go in by set_grads.
    """
    params = property(lambda self: self._params)
    grads = property(lambda self: self._grads)
    states = property(lambda self: self._states)
    copies = property(lambda self: self._copies)
    bits = property(lambda self: self._bits)
    device = property(lambda self: self._device)

    def __init__(self, params, grads, states, copies=None):
        self._params, self._states = tuple(params), tuple(states)
        self._copies = tuple(copies) if copies is not None else (None,) * len(self.params)
        if not len(self.params) == len(self.states) == len(self.copies):
            raise ValueError("params, states and copies must have the same length")
        self._device = self.params[0].device if self.params else None
        self._bits = self.states[0].bits if self.states else 32
        self._c = (_lib.AdamwTensorC * max(1, len(self.params)))()
        self._written = []        # every tensor a step writes, held here whatever becomes of the states' fields
        spans = []                # (first byte, byte past the last, tensor) of each
        for i, (w, s, h) in enumerate(zip(self.params, self.states, self.copies)):
            self._hold(i, "weight", w, torch.float32, w.numel())
            if s.bits != self.bits:
                raise ValueError("tensor %d: every state must have %d bits" % (i, self.bits))
            blocks = _fp8_blocks(w.numel())
            state = torch.float32 if self.bits == 32 else torch.uint8
            each = [("m", s.m, state, w.numel()), ("v", s.v, state, w.numel())]
            if self.bits == 8:
                each += [("m_scale", s.m_scale, torch.float32, blocks), ("v_scale", s.v_scale, torch.float32, blocks)]
            if h is not None:
                each.append(("copy", h, torch.bfloat16, w.numel()))
            for name, x, dtype, n in each:
                self._hold(i, name, x, dtype, n)
            for x in [w] + [x for _, x, _, _ in each]:
                self._written.append(x)
                if x.numel():
                    spans.append((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), i))
            c = self._c[i]
            c.w, c.m, c.v, c.n = w.data_ptr(), s.m.data_ptr(), s.v.data_ptr(), w.numel()
            if self.bits == 8:
                c.m_scales, c.v_scales = s.m_scale.data_ptr(), s.v_scale.data_ptr()
            c.copy = h.data_ptr() if h is not None else None
        spans.sort()
        for (_, end, i), (start, _, j) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError("tensors %d and %d: a weight, state or copy overlaps another" % (i, j))
        self._starts, self._spans = [start for start, _, _ in spans], spans
        self.set_grads(grads)

    def _hold(self, i, name, x, dtype, n):
        if not isinstance(x, torch.Tensor) or x.dtype != dtype or x.numel() != n or not x.is_contiguous():
            raise ValueError("tensor %d: its %s must be a contiguous %s tensor of %d elements" % (i, name, dtype, n))
        if x.device != self.device:
            raise ValueError("tensor %d: its %s is on %s, the first weight on %s" % (i, name, x.device, self.device))

    def set_grads(self, grads):
        """Other gradient tensors for the steps to come."""
        grads = tuple(grads)
        if len(grads) != len(self.params):
            raise ValueError("%d gradients for %d weights" % (len(grads), len(self.params)))
        found = []
        for i, (g, w) in enumerate(zip(grads, self._params)):
            if not isinstance(g, torch.Tensor) or g.dtype not in _OUT_KINDS:
                raise ValueError("tensor %d: its gradient must be float32 or bfloat16" % i)
            n, kind = w.numel(), _OUT_KINDS[g.dtype]
            self._hold(i, "gradient", g, g.dtype, n)
            start = g.data_ptr()
            at = bisect_left(self._starts, start + n * g.element_size()) - 1
            if n and at >= 0 and self._spans[at][1] > start:
                raise ValueError("tensors %d and %d: a gradient overlaps a weight, state or copy" % (i, self._spans[at][2]))
            found.append((start, kind))
        for c, (start, kind) in zip(self._c, found):
            c.g, c.grad = start, kind
        self._grads = grads


def _scalar(value, dtype, name, dev):
    """(host value, device address) of a number or of a one-element tensor."""
    if not isinstance(value, torch.Tensor):
        return value, None
    if value.dtype != dtype or value.numel() != 1 or value.device != dev:
        raise ValueError("%s must be a number or a one-element %s tensor on %s" % (name, dtype, dev))
    return 0, value.data_ptr()


def adamw_step(tensors, lr, step, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, rounding="rtne", seed=0,
               grad_scale=None):
    """One AdamW step (decoupled weight decay) in place on an AdamWTensors: its weights, states and copies.

    step counts from 1.  lr and step are numbers, or one-element CUDA tensors (float32, int64) that the kernel reads,
    so that a captured graph replays with values that move on.  rounding and seed are those of 8-bit states: "rtne", or
    "sr" with another seed for each step; a step on the device is added to the seed, so that every replay of a graph
    draws anew.  grad_scale: a one-element float32 CUDA tensor that every gradient is multiplied by first (clipping,
    loss scaling).
    """
    if rounding not in _lib.ROUND:
        raise ValueError("unknown rounding %r" % (rounding,))
    dev = tensors.device
    lr, lr_dev = _scalar(lr, torch.float32, "lr", dev)
    step, step_dev = _scalar(step, torch.int64, "step", dev)
    scale = None
    if grad_scale is not None:
        if not isinstance(grad_scale, torch.Tensor):
            raise ValueError("grad_scale must be a one-element torch.float32 tensor on %s" % dev)
        _, scale = _scalar(grad_scale, torch.float32, "grad_scale", dev)
    params = _lib.AdamwParamsC(lr, beta1, beta2, eps, weight_decay, step, step_dev, lr_dev, scale)
    args = (tensors._c, len(tensors.params), tensors.bits, params, _lib.ROUND[rounding], seed)
    if dev is None:
        _lib.check(_lib.mx_adamw_step(*args, None), "mx_adamw_step")       # an empty list: only the checks run
    else:
        _launch(dev.index if dev.type == "cuda" else -1, "mx_adamw_step", _lib.lib().mx_adamw_step, *args)
        _written(tensors._written)
