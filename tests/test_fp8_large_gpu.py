"""GPU parity of the 8-bit product at sizes and pitches where the tiled kernels' addresses could go wrong, and of its
kernel for large products; tests/test_fp8_path_host.py holds which kernel each shape takes."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import Fp8Tensor, fp8_gemm, fp8_quantize
from gpu_helpers import announce
from oracle import fp8
from test_fp8_gpu import assert_product, operand, tolerance

pytestmark = pytest.mark.gpu

FAR = (1 << 24) - 16                       # the largest row pitch that the tiled kernels address


def apart(q, codes_pitch, scales_pitch):
    """The same operand with rows and scale rows this far apart; what lies between is not initialised."""
    codes = torch.empty((q.codes.shape[0], codes_pitch), dtype=torch.uint8, device="cuda")[:, :q.codes.shape[1]]
    scales = torch.empty((q.scales.shape[0], scales_pitch), device="cuda")[:, :q.scales.shape[1]]
    codes.copy_(q.codes)
    scales.copy_(q.scales)
    return Fp8Tensor(codes, scales, q.k, q.fmt, q.kind)


# (m, n, k), whose rows are far apart, kernel for bf16 output.  Offsets in a 256-row tile of the large kernel pass 2^31.
FAR_SHAPES = [((130, 129, 300), "both", "mid"), ((255, 33000, 300), "a", "big"), ((256, 33000, 129), "a", "big"),
              ((4352, 2047, 300), "b", "big")]


@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("shape,which,path", FAR_SHAPES)
def test_rows_as_far_apart_as_the_tiled_kernels_go(shape, which, path, kind):
    m, n, k = shape
    rng = np.random.default_rng(m + n + k)
    a, qa = operand(m, k, "line", "e5m2", rng)
    b, qb = operand(n, k, kind, "e4m3", rng)
    wa = apart(qa, FAR, (1 << 24) + 5) if which in ("a", "both") else qa
    wb = apart(qb, FAR, 1 << 20 if kind == "tile" else (1 << 24) + 5) if which in ("b", "both") else qb
    for dtype in (torch.bfloat16, torch.float32) if path == "mid" else (torch.bfloat16,):
        announce("fp8 far rows %s %s %s %s" % (shape, which, kind, dtype))
        want = fp8_gemm(qa, qb, out_dtype=dtype)
        torch.cuda.synchronize()
        assert_product(want, a, "e5m2", b, "e4m3", kind, dtype == torch.bfloat16, (shape, kind))
        got = fp8_gemm(wa, wb, out_dtype=dtype)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_than_2_to_24_rows(dtype):
    """Every row is the one that the product of its own million rows gives, and the first and last are the oracle's."""
    m, n, k = (1 << 24) + 77, 24, 100
    rng = np.random.default_rng(20)
    b, qb = operand(n, k, "tile", "e4m3", rng)
    gen = torch.Generator(device="cuda").manual_seed(20)
    codes = torch.randint(0, 0x7F, (m, 128), dtype=torch.uint8, device="cuda", generator=gen)
    codes[:, k:] = 0
    scales = torch.rand((1, m), device="cuda", generator=gen) + 0.5
    announce("fp8 product of 2^24 rows %s" % dtype)
    got = fp8_gemm(Fp8Tensor(codes, scales, k), qb, out_dtype=dtype)
    torch.cuda.synchronize()
    part = 1 << 20
    for at in range(0, m, part):
        q = Fp8Tensor(codes[at:at + part], scales[:, at:at + part].contiguous(), k)
        assert torch.equal(got[at:at + part], fp8_gemm(q, qb, out_dtype=dtype))
    for rows in (slice(0, 300), slice(m - 300, m)):
        a = codes[rows].cpu().numpy(), scales[:, rows].cpu().numpy()
        assert_product(got[rows], a, "e4m3", b, "e4m3", "tile", dtype == torch.bfloat16, "rows %s" % (rows,))


# (m, n, k) of the kernel for large products: edge tiles on either side, 9 to 112 K blocks, odd and even, one round of the
# chip and several
BIG = [(257, 24001, 1300), (4000, 8101, 1100), (8192, 8190, 4000), (500, 17000, 14336), (4351, 2047, 8001)]


def chunks(m, n):
    """(first column, columns) that cover n columns so that each part has 257 to 512 tiles of 128 x 128: it runs whole, on
    the kernel for mid-sized products.  First columns are multiples of 128, where tile scales begin."""
    tm, tn = -(-m // 128), -(-n // 128)
    count = -(-tn // (512 // tm))
    width = -(-tn // count)
    starts = [min(i * width, tn - width) for i in range(count)]
    return [(128 * t, min(128 * width, n - 128 * t)) for t in starts]


def device_operand(lines, k, kind, fmt, gen, inside=False):
    """Codes of every finite value, scales over six binades; inside: in larger buffers, NaN around and between the rows."""
    kb = -(-k // 128)
    top = fp8.FORMATS[fmt][3]
    codes = torch.full((lines + 2, kb * 128 + 32), 0x7F, dtype=torch.uint8, device="cuda")[1:-1, 16:-16]
    codes.random_(0, 2 * top + 2, generator=gen)
    codes.copy_(torch.where(codes > top, codes - (top + 1) + 128, codes))
    codes[:, k:] = 0
    rows, cols = (kb, lines) if kind == "line" else (-(-lines // 128), kb)
    scales = torch.full((rows + 2, cols + 3), float("nan"), device="cuda")[1:-1, 1:-2]
    scales.copy_(torch.exp2(6 * torch.rand((rows, cols), generator=gen, device="cuda") - 3))
    if inside:
        return Fp8Tensor(codes, scales, k, fmt, kind)
    return Fp8Tensor(codes.contiguous(), scales.contiguous(), k, fmt, kind)


def some(size, count, rng):
    """Indices: the first and last 20, the ones around each border of 128 up to 1024, and random ones."""
    near = [i + d for i in range(128, 1025, 128) for d in (-1, 0)]
    pick = np.concatenate([np.arange(20), np.arange(size - 20, size), near, rng.integers(0, size, count)])
    return np.unique(pick[pick < size])


def host_lines(q, lines):
    """The oracle's (codes, scales) of some lines of an operand, scales as a line operand holds them."""
    at = torch.from_numpy(lines).cuda()
    scales = q.scales[:, at] if q.kind == "line" else q.scales[at // 128].t()
    return q.codes[at].cpu().numpy(), scales.contiguous().cpu().numpy()


def check_some(got, qa, qb, rng, what):
    rows, cols = some(qa.lines, 200, rng), some(qb.lines, 400, rng)
    part = got[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()]
    return assert_product(part, host_lines(qa, rows), qa.fmt, host_lines(qb, cols), qb.fmt, "line", True, what)


def columns_of(q, at, n):
    scales = q.scales[:, at:at + n] if q.kind == "line" else q.scales[at // 128:-(-(at + n) // 128)]
    return Fp8Tensor(q.codes[at:at + n], scales, q.k, q.fmt, q.kind)


@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("af,bf", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", BIG)
def test_large_products(m, n, k, af, bf, kind):
    """Sampled rows and columns against the oracle; the whole output, bit for bit, against a second run and against the
    kernel for mid-sized products, which adds the same blocks in the same order."""
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    qa, qb = device_operand(m, k, "line", af, gen), device_operand(n, k, kind, bf, gen)
    announce("fp8 large %dx%dx%d %s %s %s" % (m, n, k, af, bf, kind))
    got = fp8_gemm(qa, qb, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    print("err/G %.3g" % check_some(got, qa, qb, np.random.default_rng(m), (m, n, k, af, bf, kind)))
    assert torch.equal(fp8_gemm(qa, qb, out_dtype=torch.bfloat16), got)
    for at, width in chunks(m, n):
        assert torch.equal(fp8_gemm(qa, columns_of(qb, at, width), out_dtype=torch.bfloat16), got[:, at:at + width])


@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("af,bf", [("e4m3", "e4m3"), ("e5m2", "e4m3")])
@pytest.mark.parametrize("m,n,k", [BIG[0], BIG[1]])
def test_large_products_inside_larger_buffers(m, n, k, af, bf, kind):
    """Operands between NaN codes and scales, output rows at several alignments and odd pitches: the numbers are the same
    and nothing around them changes."""
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    qa, qb = device_operand(m, k, "line", af, gen, True), device_operand(n, k, kind, bf, gen, True)
    packed = [Fp8Tensor(q.codes.contiguous(), q.scales.contiguous(), k, q.fmt, q.kind) for q in (qa, qb)]
    announce("fp8 large in buffers %dx%dx%d %s %s %s" % (m, n, k, af, bf, kind))
    want = fp8_gemm(*packed, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    check_some(want, *packed, np.random.default_rng(m), (m, n, k))
    for left, pitch in ((0, n), (1, n + 2 + n % 2), (8, n + 16 + (-n) % 8), (3, n + 4 + n % 2)):
        buf = torch.full((m + 2, pitch + 8), -3.0, dtype=torch.bfloat16, device="cuda")
        got = fp8_gemm(qa, qb, out=buf[1:-1, left:left + n])
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        got.fill_(-3.0)
        assert bool((buf == -3.0).all())


@pytest.mark.parametrize("block", [0, 4, 8])
@pytest.mark.parametrize("kind", ["line", "tile"])
def test_large_products_with_nan_and_inf(kind, block):
    """NaN and Inf in one block of single lines (of 128 lines with a tile scale), first, middle and last, reach the rows
    and columns of those lines and nothing else: all codes are positive, so no Inf meets its negative."""
    m, n, k = 4000, 8101, 1100
    gen = torch.Generator(device="cuda").manual_seed(21)
    qa, qb = device_operand(m, k, "line", "e5m2", gen), device_operand(n, k, kind, "e4m3", gen)
    for q in (qa, qb):
        q.codes &= 0x7F
        q.codes[:, 128 * block:k if block == 8 else 128 * (block + 1)].clamp_(min=1)
    clean = fp8_gemm(qa, qb, out_dtype=torch.bfloat16)
    want = clean.clone()
    qa.codes[5, 128 * block] = 0x7C                   # E5M2 Inf
    qa.scales[block, 255] = float("inf")
    qa.scales[block, 3999] = float("nan")
    want[[5, 255]], want[3999] = float("inf"), float("nan")
    if kind == "line":
        qb.scales[block, 8100] = float("nan")
        want[:, 8100] = float("nan")
    else:
        qb.scales[1, block] = float("nan")            # lines 128 .. 255, the second half of a 256-wide tile
        want[:, 128:256] = float("nan")
    qb.codes[300, 128 * block] = 0x7F                 # E4M3 NaN
    want[:, 300] = float("nan")
    announce("fp8 large nan and inf %s block %d" % (kind, block))
    got = fp8_gemm(qa, qb, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0, posinf=1e38), want.nan_to_num(nan=0.0, posinf=1e38))


@pytest.mark.parametrize("kind,fmt", [("tile", "e4m3"), ("line", "e5m2")])
def test_large_products_of_normal_data(kind, fmt):
    """Cast normal data (the second, as an E5M2 gradient): off by at most 2^-14 of the row-column magnitudes' sum before
    the rounding to bf16, and in norm by that rounding's, at most 2^-8 / sqrt 3."""
    m, n, k = 4096, 8192, 4096
    gen = torch.Generator(device="cuda").manual_seed(22)
    x, w = (torch.randn(size, generator=gen, device="cuda").bfloat16() for size in ((m, k), (n, k)))
    qa, qb = fp8_quantize(x, fmt=fmt)["row"], fp8_quantize(w, kind=kind)["row"]
    announce("fp8 large normal data %s %s" % (kind, fmt))
    got = fp8_gemm(qa, qb, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    rng = np.random.default_rng(22)
    rows, cols = some(m, 500, rng), some(n, 500, rng)
    c, g = fp8.gemm_ref(host_lines(qa, rows), fmt, host_lines(qb, cols), "e4m3", "line")
    part = got[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()].double().cpu().numpy()
    assert np.all(np.abs(part - c) <= 2.0 ** -14 * g + 2.0 ** -8 * (np.abs(c) + 2.0 ** -14 * g))
    assert np.linalg.norm(part - c) <= 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(c)


# few rows, mid (whole and in parts), large
SMALL_SCALES = [(3, 300, 1100), (20, 40, 700), (300, 300, 300), (200, 260, 4100), (4352, 2047, 300)]


@pytest.mark.parametrize("low", [-134, -145, -155])
@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("m,n,k", SMALL_SCALES)
def test_scales_whose_product_is_not_a_normal_number(m, n, k, kind, low):
    """Products of scales around 2^low, within 2^6: a product is rounded to a multiple of 2^-149, off by at most 2^-150,
    and so is each of the at most K / 128 + 9 additions whose result is that small (eight waves' sums among them); a bf16
    result that small is off by half of bf16's least step 2^-133."""
    rng = np.random.default_rng(m + n - low)
    a, qa = operand(m, k, "line", "e5m2", rng, 2.0 ** (low // 2))
    b, qb = operand(n, k, kind, "e4m3", rng, 2.0 ** (low - low // 2))
    kb = a[0].shape[1] // 128
    c, g = fp8.gemm_ref(a, "e5m2", b, "e4m3", kind)
    codes = np.abs(fp8.decode(a[0], "e5m2")) @ np.abs(fp8.decode(b[0], "e4m3")).T
    for bf16 in (False, True):
        announce("fp8 small scales %dx%dx%d %s 2^%d %s" % (m, n, k, kind, low, "bf16" if bf16 else "fp32"))
        got = fp8_gemm(qa, qb, torch.bfloat16 if bf16 else torch.float32)
        torch.cuda.synchronize()
        tol = tolerance(c, g, kb, bf16) + (2.0 ** -150 * codes + (kb + 9) * 2.0 ** -150) * (1 + bf16 * 2.0 ** -8)
        tol += bf16 * 2.0 ** -134
        assert np.all(np.abs(got.double().cpu().numpy() - c) <= tol)
