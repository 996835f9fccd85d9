"""GPU parity of the 8-bit cast and product against the oracle: codes and scales byte for byte, products within the
float32 accumulation's bound, padding and neighbouring memory untouched."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import Fp8Tensor, empty_fp8, fp8_gemm, fp8_quantize, synth
from gpu_helpers import announce, assert_bytes_equal, to_gpu_bits
from oracle import fp8

pytestmark = pytest.mark.gpu


def bits_of(x):
    return synth.f32_to_bf16_bits(x.astype(np.float32))


def rough(rows, cols, rng):
    """Normal values with outlier columns, a zero row and column, and rows of very small and very large values."""
    x = rng.standard_normal((rows, cols))
    x[:, rng.integers(0, cols, max(1, cols // 100))] *= 50.0
    x[rng.integers(0, rows, 1 + rows // 50)] *= 2.0 ** -120
    x[rng.integers(0, rows, 1 + rows // 50)] *= 2.0 ** 100
    x[rows // 2] = 0.0
    x[:, cols // 3] = 0.0
    return bits_of(x)


def check(q, want, what):
    for axis, (codes, scales) in want.items():
        assert_bytes_equal(q[axis].codes.cpu().numpy(), codes, what + " " + axis + " codes")
        assert_bytes_equal(q[axis].scales.cpu().numpy().view(np.uint32), scales.view(np.uint32), what + " " + axis + " scales")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (2, 120), (127, 136), (128, 128), (129, 264), (300, 1000), (1001, 512)])
def test_cast_matches_the_oracle(rows, cols, kind, fmt):
    bits = rough(rows, cols, np.random.default_rng(rows * 7 + cols))
    x = to_gpu_bits(bits).view(torch.bfloat16)
    for axis in ("row", "col", "both"):
        announce("fp8 cast %dx%d %s %s %s" % (rows, cols, kind, fmt, axis))
        q = fp8_quantize(x, axis=axis, kind=kind, fmt=fmt)
        torch.cuda.synchronize()
        assert sorted(q) == sorted(["row", "col"] if axis == "both" else [axis])
        check(q, fp8.quantize_ref(bits, axis, kind, fmt), "%s %s" % (kind, fmt))


@pytest.mark.parametrize("kind", ["line", "tile"])
def test_every_bf16_value(kind):
    """All 65536 bf16 patterns, Inf and NaN with every payload among them, as blocks of like exponents and shuffled."""
    rng = np.random.default_rng(5)
    allv = np.arange(65536, dtype=np.uint16).reshape(512, 128)
    for name, bits in (("ordered", allv), ("shuffled", rng.permutation(allv.reshape(-1)).reshape(512, 128)),
                       ("pairs", np.concatenate([allv, np.full((512, 128), 0x4000, np.uint16)], axis=1))):
        for fmt in ("e4m3", "e5m2"):
            announce("fp8 every bf16 %s %s %s" % (name, kind, fmt))
            q = fp8_quantize(to_gpu_bits(bits).view(torch.bfloat16), axis="both", kind=kind, fmt=fmt)
            want = fp8.quantize_ref(bits, "both", kind, fmt)
            for axis in want:
                assert_bytes_equal(q[axis].codes.cpu().numpy(), want[axis][0], name + " codes")
                got, ref = q[axis].scales.cpu().numpy(), want[axis][1]
                assert np.array_equal(got, ref, equal_nan=True)


def test_cast_into_larger_buffers():
    """A strided input, outputs inside larger buffers: nothing beside the outputs' own lines changes."""
    rng = np.random.default_rng(6)
    rows, cols = 150, 200
    big = to_gpu_bits(rough(rows + 3, cols + 48, rng)).view(torch.bfloat16)
    x = big[2:2 + rows, 16:16 + cols]
    bits = x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    for kind in ("line", "tile"):
        announce("fp8 strided " + kind)
        bufs, outs = [], []
        for lines, k in ((rows, cols), (cols, rows)):
            like = empty_fp8(lines, k, "cpu", kind=kind)
            codes = torch.full((lines + 2, like.codes.shape[1] + 16), 0xA5, dtype=torch.uint8, device="cuda")
            scales = torch.full((like.scales.shape[0] + 2, like.scales.shape[1] + 5), -7.0, device="cuda")
            bufs.append((codes, scales))
            outs.append(Fp8Tensor(codes[1:1 + lines, :like.codes.shape[1]],
                                  scales[1:1 + like.scales.shape[0], 2:2 + like.scales.shape[1]], k, "e4m3", kind))
        q = fp8_quantize(x, axis="both", kind=kind, row_out=outs[0], col_out=outs[1])
        torch.cuda.synchronize()
        assert q["row"] is outs[0]
        check(q, fp8.quantize_ref(bits, "both", kind, "e4m3"), "strided " + kind)
        for (codes, scales), o in zip(bufs, outs):
            o.codes.fill_(0xA5)
            o.scales.fill_(-7.0)
            assert bool((codes == 0xA5).all()) and bool((scales == -7.0).all())


def operand(lines, k, kind, fmt, rng, scale=1.0):
    """An operand on both sides: codes of every finite value but mostly moderate ones, scales over some binades."""
    kb = -(-k // 128)
    top = fp8.FORMATS[fmt][3]
    codes = np.zeros((lines, kb * 128), dtype=np.uint8)
    codes[:, :k] = rng.integers(0, top + 1, (lines, k)) | (rng.integers(0, 2, (lines, k)) << 7)
    shape = (kb, lines) if kind == "line" else (-(-lines // 128), kb)
    scales = (scale * np.exp2(rng.uniform(-3, 3, shape))).astype(np.float32)
    return (codes, scales), Fp8Tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), k, fmt, kind)


def tolerance(c, g, kb, bf16):
    """What a product may be off by.

    fp32 output: the matrix core adds 128 exact products in float32, losing at most one unit in the last place (2^-23)
    of the sum of magnitudes for each; the product of the scales, and then each block's fused multiply-add, round once
    (2^-24).

    bf16 output: the 8-bit matrix instruction aligns the products of each 8 neighbouring k to the largest and drops what
    lies below 2^-13 of it.  The largest loses nothing, each of the other 7 less than 2^-13 of it, and the largest is at
    most the run's sum of magnitudes: 7 * 2^-13 of it.  The 16 runs' sums add in float32 (16 * 2^-23), and the rounding
    to bf16 is half a step, 2^-8."""
    if not bf16:
        return (128 * 2.0 ** -23 + (kb + 2) * 2.0 ** -24) * g
    tol = (7 * 2.0 ** -13 + 16 * 2.0 ** -23 + (kb + 2) * 2.0 ** -24) * g
    return tol + 2.0 ** -8 * (np.abs(c) + tol)


def assert_product(got, a, a_fmt, b, b_fmt, kind, bf16, what):
    c, g = fp8.gemm_ref(a, a_fmt, b, b_fmt, kind)
    tol = tolerance(c, g, a[0].shape[1] // 128, bf16)
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - c)
    bad = np.argwhere(~(err <= tol))
    assert not bad.size, (what, len(bad), tuple(bad[0]), got[tuple(bad[0])].item(), c[tuple(bad[0])])
    return float((err / np.maximum(g, 1e-300)).max())


def test_bf16_output_on_normal_data():
    """On cast normal data the 8-bit instruction's dropped parts stay far inside a bf16 rounding: the result before
    rounding is off by at most 2^-14 of the row-column magnitudes' sum (a product 2^-13 below the largest of 8 is rare,
    and each drop is a fraction of it), so the norm of the error is that of the bf16 rounding, at most 2^-8 / sqrt 3."""
    rng = np.random.default_rng(10)
    x, w = bits_of(rng.standard_normal((512, 2048))), bits_of(0.02 * rng.standard_normal((512, 2048)))
    a, b = fp8.quantize_lines(fp8.bf16_values(x), "line", "e4m3"), fp8.quantize_lines(fp8.bf16_values(w), "tile", "e4m3")
    qa = fp8_quantize(to_gpu_bits(x).view(torch.bfloat16))["row"]
    qb = fp8_quantize(to_gpu_bits(w).view(torch.bfloat16), kind="tile")["row"]
    announce("fp8 normal data")
    c, g = fp8.gemm_ref(a, "e4m3", b, "e4m3", "tile")
    got = fp8_gemm(qa, qb, out_dtype=torch.bfloat16).float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - c) <= 2.0 ** -14 * g + 2.0 ** -8 * (np.abs(c) + 2.0 ** -14 * g))
    assert np.linalg.norm(got - c) <= 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(c)


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 1000, 300), (2, 130, 129), (5, 4096, 512), (15, 129, 4000), (16, 512, 1024),
          (17, 65, 257), (31, 1003, 640), (33, 300, 1000), (64, 256, 14336), (65, 500, 384), (100, 1, 700),
          (128, 128, 128), (129, 127, 255), (255, 257, 600), (256, 256, 256), (300, 1003, 1001), (512, 768, 640),
          (700, 520, 2000), (1000, 1300, 385),
          (4200, 4300, 300), (4000, 8100, 300), (256, 33000, 128), (500, 17000, 200), (40, 200, 9000), (300, 500, 4100)]


@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_matches_the_oracle(m, n, k, kind):
    rng = np.random.default_rng(m * 31 + n * 7 + k)
    a, qa = operand(m, k, "line", "e4m3", rng)
    b, qb = operand(n, k, kind, "e4m3", rng, 0.01)
    for dtype in (torch.float32, torch.bfloat16):
        announce("fp8 product %dx%dx%d %s %s" % (m, n, k, kind, dtype))
        got = fp8_gemm(qa, qb, out_dtype=dtype)
        torch.cuda.synchronize()
        e = assert_product(got, a, "e4m3", b, "e4m3", kind, dtype == torch.bfloat16, (m, n, k, kind))
        print("err/G %.3g" % e)


@pytest.mark.parametrize("af,bf", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(3, 260, 1000), (40, 200, 512), (200, 140, 700), (600, 780, 1100)])
def test_product_formats(m, n, k, af, bf):
    rng = np.random.default_rng(m + n + k)
    for kind in ("line", "tile"):
        a, qa = operand(m, k, "line", af, rng, 1e-3)
        b, qb = operand(n, k, kind, bf, rng)
        announce("fp8 product %dx%dx%d %s %s %s" % (m, n, k, af, bf, kind))
        got = fp8_gemm(qa, qb)
        torch.cuda.synchronize()
        assert_product(got, a, af, b, bf, kind, False, (m, n, k, af, bf, kind))


@pytest.mark.parametrize("m,n,k", [(1, 300, 512), (20, 77, 300), (150, 300, 256), (700, 700, 700)])
def test_product_into_larger_buffers(m, n, k):
    """Operands and output with row pitches of their own, output rows at every alignment: the numbers are the same and
    nothing beside the M x N outputs changes, before, behind or between the rows."""
    rng = np.random.default_rng(m * n)
    for kind in ("line", "tile"):
        _, qa = operand(m, k, "line", "e4m3", rng)
        _, qb = operand(n, k, kind, "e4m3", rng)

        def inside(q):
            codes = torch.full((q.codes.shape[0] + 2, q.codes.shape[1] + 32), 0x7F, dtype=torch.uint8, device="cuda")
            scales = torch.full((q.scales.shape[0] + 2, q.scales.shape[1] + 3), float("nan"), device="cuda")
            c, s = codes[1:-1, 16:-16], scales[1:-1, 1:-2]
            c.copy_(q.codes)
            s.copy_(q.scales)
            return Fp8Tensor(c, s, q.k, q.fmt, q.kind)
        wa, wb = inside(qa), inside(qb)
        for dtype in (torch.float32, torch.bfloat16):
            want = fp8_gemm(qa, qb, out_dtype=dtype)
            for left, pitch in ((0, n), (1, n + 1), (4, n + 8 + (-n) % 8), (8, n + 16 + (-n) % 8)):
                announce("fp8 product in buffers %dx%dx%d %s %s at %d" % (m, n, k, kind, dtype, left))
                buf = torch.full((m + 2, pitch + 8), -3.0, dtype=dtype, device="cuda")
                got = fp8_gemm(wa, wb, out=buf[1:-1, left:left + n])
                torch.cuda.synchronize()
                assert torch.equal(got, want)
                got.fill_(-3.0)
                assert bool((buf == -3.0).all())


def test_nan_blocks_reach_only_their_rows_and_columns():
    rng = np.random.default_rng(8)
    for m, n, k in ((4, 200, 384), (200, 300, 384), (600, 600, 512)):
        x = rng.standard_normal((m, k))
        x[1, 200] = np.nan
        w = rng.standard_normal((n, k))
        w[5, 3] = np.inf
        qx = fp8_quantize(to_gpu_bits(bits_of(x)).view(torch.bfloat16))["row"]
        qw = fp8_quantize(to_gpu_bits(bits_of(w)).view(torch.bfloat16))["row"]
        announce("fp8 nan blocks %d %d %d" % (m, n, k))
        c = fp8_gemm(qx, qw)
        bad = torch.zeros_like(c, dtype=torch.bool)
        bad[1], bad[:, 5] = True, True
        assert torch.equal(torch.isnan(c), bad)


@pytest.mark.parametrize("m,n,k", [(40, 33, 300), (70, 20, 130)])
def test_rows_far_apart(m, n, k):
    """Operand rows and scale rows 2^24 bytes and floats apart: the same numbers as close together, with offsets that
    pass 31 bits."""
    rng = np.random.default_rng(16)
    for kind in ("line", "tile"):
        _, qa = operand(m, k, "line", "e4m3", rng)
        _, qb = operand(n, k, kind, "e4m3", rng)

        def apart(q):
            codes = torch.zeros((q.codes.shape[0], 1 << 24), dtype=torch.uint8, device="cuda")[:, :q.codes.shape[1]]
            codes.copy_(q.codes)
            scales = torch.zeros((q.scales.shape[0], 1 << 24), device="cuda")[:, :q.scales.shape[1]]
            scales.copy_(q.scales)
            return Fp8Tensor(codes, scales, q.k, q.fmt, q.kind)
        announce("fp8 rows far apart %s" % kind)
        for dtype in (torch.float32, torch.bfloat16):
            got = fp8_gemm(apart(qa), apart(qb), out_dtype=dtype)
            torch.cuda.synchronize()
            assert_product(got, (qa.codes.cpu().numpy(), qa.scales.cpu().numpy()), "e4m3",
                           (qb.codes.cpu().numpy(), qb.scales.cpu().numpy()), "e4m3", kind, dtype == torch.bfloat16,
                           (m, n, k, kind))


def test_cast_of_a_large_matrix():
    """More than 2^31 elements: the last rows and columns of each output are those of the same rows cast alone."""
    rows, cols = 131072 + 128, 16400
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x[-256:] = torch.randn((256, cols), generator=gen, device="cuda").bfloat16()
    announce("fp8 cast of a large matrix")
    q = fp8_quantize(x, axis="both")
    tail = fp8_quantize(x[-256:].contiguous(), axis="both")
    assert torch.equal(q["row"].codes[-256:], tail["row"].codes) and torch.equal(q["row"].scales[:, -256:], tail["row"].scales)
    assert torch.equal(q["col"].codes[:, -256:], tail["col"].codes) and torch.equal(q["col"].scales[-2:], tail["col"].scales)
    assert int(q["row"].codes[:1000].max()) == 0 and int(q["col"].codes[-1, :1000].max()) == 0


def test_split_products_at_once_and_replayed():
    """Products whose K is split over workgroups: two at once on two streams, each with its workspace, and two captured
    graphs replayed in turn and at once, with eager products between: every result is the eager one's, bit for bit.  A
    smaller or no workspace gives fewer parts and the same numbers within the accumulation bound."""
    from block_scaled_fp4_hadamard_amd import _lib
    rng = np.random.default_rng(17)
    m, n, k = 300, 500, 8192
    assert _lib.mx_fp8_gemm_workspace(m, n, k, 1) > 4 * m * n
    ops = [(operand(m, k, "line", "e4m3", rng), operand(n, k, "tile", "e4m3", rng)) for _ in range(2)]
    want = [[fp8_gemm(a[1], b[1], out_dtype=d) for a, b in ops] for d in (torch.bfloat16, torch.float32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    announce("fp8 split products on two streams")
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                fp8_gemm(ops[i][0][1], ops[i][1][1], out=outs[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0][0]) and torch.equal(outs[1], want[0][1])
    announce("fp8 split products in graphs")
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fp8_gemm(ops[i][0][1], ops[i][1][1], out=outs[i])
        graphs.append(g)
    for turn in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        again = fp8_gemm(ops[turn % 2][0][1], ops[turn % 2][1][1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0][0]) and torch.equal(outs[1], want[0][1])
        assert torch.equal(again, want[1][turn % 2])
    (a, qa), (b, qb) = ops[0]
    full = _lib.mx_fp8_gemm_workspace(m, n, k, 0)
    for size in (full // 2, 0):
        announce("fp8 split product with %d bytes" % size)
        space = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        c = torch.empty((m, n), device="cuda")
        _lib.check(_lib.mx_fp8_gemm(qa.c_struct(), 0, qb.c_struct(), 0, 1, m, n, k, c.data_ptr(), n, 0,
                                    space.data_ptr() if size else None, size, torch.cuda.current_stream().cuda_stream),
                   "mx_fp8_gemm")
        torch.cuda.synchronize()
        assert_product(c, a, "e4m3", b, "e4m3", "tile", False, size)


def test_empty_products():
    a, b = empty_fp8(0, 128, "cuda"), empty_fp8(5, 128, "cuda")
    assert fp8_gemm(a, b).shape == (0, 5)
    assert fp8_quantize(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"))["row"].codes.shape == (0, 128)


def test_streams_and_graph():
    """Two calls at once on two streams, and a captured cast and product replayed with new inputs: each result is the
    eager one's, bit for bit, with eager work and synchronizations between the replays."""
    rng = np.random.default_rng(9)
    xs = [torch.from_numpy(rng.standard_normal((300, 640)).astype(np.float32)).cuda().bfloat16() for _ in range(4)]
    w = torch.from_numpy(rng.standard_normal((500, 640)).astype(np.float32)).cuda().bfloat16()
    qw = fp8_quantize(w, kind="tile")["row"]
    want = [fp8_gemm(fp8_quantize(x)["row"], qw) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                got[i] = fp8_gemm(fp8_quantize(xs[i])["row"], qw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = xs[0].clone()
    q = empty_fp8(300, 640, "cuda")
    c = torch.empty((300, 500), device="cuda")
    announce("fp8 graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8_quantize(x, row_out=q)
        fp8_gemm(q, qw, out=c)
    for i in (1, 2, 3, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want[i])
        assert torch.equal(fp8_gemm(fp8_quantize(xs[i])["row"], qw), want[i])


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 650), (20, 9000, 130), (40, 300, 1100), (200, 130, 128)])
def test_infinities_stay_infinite(M, N, K, kind, bf16):
    """An E5M2 Inf code or an Inf scale in a line's last block gives that line Inf, a NaN scale NaN, the others nothing,
    whatever the number of blocks.  All values are positive, so that no Inf meets its negative."""
    rng = np.random.default_rng(M + N)
    (ac, asc), _ = operand(M, K, "line", "e5m2", rng)
    (bc, bsc), _ = operand(N, K, kind, "e4m3", rng)
    ac &= 0x7F
    bc &= 0x7F
    bc[:, K - 1] = 0x38            # 1
    ac[:3, K - 1] = 0x3C           # 1
    clean = ac.copy(), asc.copy()
    ac[0, K - 1] = 0x7C
    asc[-1, 1], asc[-1, 2] = np.inf, np.nan
    a = Fp8Tensor(torch.from_numpy(ac).cuda(), torch.from_numpy(asc).cuda(), K, "e5m2", "line")
    b = Fp8Tensor(torch.from_numpy(bc).cuda(), torch.from_numpy(bsc).cuda(), K, "e4m3", kind)
    announce("fp8 infinities %dx%dx%d %s %s" % (M, N, K, kind, "bf16" if bf16 else "fp32"))
    got = fp8_gemm(a, b, torch.bfloat16 if bf16 else torch.float32)
    torch.cuda.synchronize()
    assert bool((got[:2] == float("inf")).all())
    assert bool(got[2].isnan().all())
    if M > 3:
        rest = tuple(np.ascontiguousarray(x) for x in (clean[0][3:], clean[1][:, 3:]))
        assert_product(got[3:], rest, "e5m2", (bc, bsc), "e4m3", kind, bf16, "rest")


@pytest.mark.parametrize("bf16", [False, True], ids=["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("M", [1, 16, 17, 32])
@pytest.mark.parametrize("N", [4095, 5001, 10241, 14335, 20490, 28673])
def test_few_rows_over_all_widths(M, N, kind, bf16):
    """Every number of column fragments that the kernel for few rows takes, with a part-filled last one."""
    K = 300 + 1100 * (N % 2)
    rng = np.random.default_rng(M * N)
    a, qa = operand(M, K, "line", "e4m3", rng)
    b, qb = operand(N, K, kind, "e5m2", rng)
    announce("fp8 few %dx%dx%d %s %s" % (M, N, K, kind, "bf16" if bf16 else "fp32"))
    buf = torch.full((M + 1, N + 5), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    got = fp8_gemm(qa, qb, out=buf[:M, :N])
    torch.cuda.synchronize()
    assert_product(got, a, "e4m3", b, "e5m2", kind, bf16, "few")
    assert bool((buf[M] == 7.0).all()) and bool((buf[:, N:] == 7.0).all())
