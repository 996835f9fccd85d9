"""GPU parity of the 8-bit product at sizes and pitches where the tiled kernels' addresses could go wrong, and of its
kernel for large products; tests/test_fp8_path_host.py holds which kernel each shape takes."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import Fp8Tensor, fp8_gemm
from gpu_helpers import announce
from test_fp8_gpu import assert_product, operand

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
