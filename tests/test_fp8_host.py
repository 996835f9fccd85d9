"""Host side of the 8-bit operands and the AdamW step: pins of their oracles, and what the entry points refuse (CPU only:
no call here reaches a kernel)."""
import gc
import math
import weakref
from fractions import Fraction

import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import AdamWState, AdamWTensors, Fp8Tensor, _lib, adamw_step, api, empty_fp8, fp8_gemm, fp8_quantize
from oracle import adamw, fp8

FAKE = 0x10000          # an aligned non-null address; validation never dereferences it
TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ---- oracle pins

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_levels_and_rounding_agree_with_torch(fmt):
    """Every finite code decodes as torch decodes it, and the nearest-level search rounds as torch's cast does, on every
    midpoint, both neighbours of it and random values inside the range."""
    table = fp8.levels(fmt)
    codes = torch.arange(len(table), dtype=torch.uint8)
    assert np.array_equal(table, codes.view(TORCH[fmt]).double().numpy())
    mid = ((table[1:] + table[:-1]) / 2).astype(np.float32)
    rng = np.random.default_rng(1)
    x = np.concatenate([table, mid, np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(0)),
                        rng.uniform(0, table[-1], 20000), np.exp2(rng.uniform(-20, np.log2(table[-1]), 20000))])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(TORCH[fmt]).view(torch.uint8).numpy()
    assert np.array_equal(fp8.nearest_code(x.astype(np.float64), table), want)


@pytest.mark.parametrize("kind", ["line", "tile"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_cast_is_within_half_a_step(kind, fmt):
    """A block's largest value gets the top code; every decoded value is within half a step of the format plus the three
    float32 roundings of s, r and x r; the column output is the transpose's row output."""
    rng = np.random.default_rng(2)
    bits = (rng.standard_normal((200, 264)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    x = fp8.bf16_values(bits)
    q = fp8.quantize_ref(bits, "both", kind, fmt)
    codes, scales = q["row"]
    assert codes.shape == (200, 384) and not codes[:, 264:].any()
    v = fp8.values(codes, scales, kind, fmt)[:, :264]
    s = np.repeat(scales.T if kind == "line" else np.repeat(scales, 128, axis=0)[:200], 128, axis=1)[:, :264]
    half = 2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3
    least = 2.0 ** -10 if fmt == "e4m3" else 2.0 ** -17          # half the subnormal step
    assert np.all(np.abs(v - x) <= (half + 2.0 ** -21) * np.abs(x) + least * (1 + 2.0 ** -20) * s)
    top = fp8.FORMATS[fmt][3]
    assert np.all((codes & 0x7F).reshape(200, 3, 128).max(axis=2)[:, :2].max(axis=0) == top)
    t = fp8.quantize_lines(np.ascontiguousarray(x.T), kind, fmt)
    assert np.array_equal(q["col"][0], t[0]) and np.array_equal(q["col"][1], t[1])


def test_special_blocks():
    x = np.zeros((3, 256), dtype=np.float32)
    x[0, 5] = np.inf
    x[1, 200] = np.nan
    x[2, 0], x[2, 1] = -2.0 ** -133, 0.0
    codes, s = fp8.quantize_lines(x, "line", "e4m3")
    assert np.isnan(s[0, 0]) and np.isnan(s[1, 1]) and not codes[:2].any()
    assert s[0, 1] == s[0, 2] == np.float32(2.0 ** -126)
    assert codes[2, 0] == 0x84 and codes[2, 1] == 0        # -2^-133 2^126 = -2^-7: four subnormal steps of 2^-9


def test_gemm_reference_by_hand():
    """One block of exact small numbers, against Fractions."""
    a = (np.array([[0x38, 0xB8, 0x40] + [0] * 125], dtype=np.uint8), np.array([[0.5]], dtype=np.float32))
    b = (np.array([[0x38, 0x30, 0x01] + [0] * 125], dtype=np.uint8), np.array([[3.0]], dtype=np.float32))
    c, g = fp8.gemm_ref(a, "e4m3", b, "e4m3", "line")
    one = Fraction(1) - Fraction(1, 2) + 2 * Fraction(1, 512)
    assert Fraction(float(c[0, 0])) == one * Fraction(3, 2)
    assert Fraction(float(g[0, 0])) == (one + 1) * Fraction(3, 2)


def test_adamw_against_torch():
    """32-bit moments over 30 steps against torch.optim.AdamW in float64.  A step multiplies and adds each float32 once
    per operation, so m and v stay within a few 2^-24 of theirs and w within the 30 steps' roundings."""
    rng = np.random.default_rng(3)
    w = rng.standard_normal(1000).astype(np.float32)
    m, v = np.zeros(1000, np.float32), np.zeros(1000, np.float32)
    p = torch.nn.Parameter(torch.from_numpy(w.astype(np.float64)))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    for t in range(1, 31):
        g = rng.standard_normal(1000).astype(np.float32)
        w, m, v = adamw.update(w, g, m, v, adamw.coefficients(1e-2, 0.9, 0.99, 1e-8, 0.1, t))
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
    err = np.abs(w - p.detach().numpy())
    # per step: w is rounded at its own size (2^-24 |w|), the update (at most ~1e-2) within 8 roundings of 2^-24
    assert err.max() <= 30 * 2.0 ** -24 * (3 * np.abs(w).max() + 8e-2)


def test_e5m3_is_float16_without_its_tail():
    codes = np.arange(0xF8, dtype=np.uint16)
    assert np.array_equal(adamw.E5M3, (codes << 7).view(np.float16).astype(np.float64))


def test_state_codes():
    """Nearest: half a step; stochastic: unbiased and never off by a whole step; v above 0 keeps a code above 0."""
    rng = np.random.default_rng(4)
    x = np.exp2(rng.uniform(-30, 0, 1280)).astype(np.float32)
    for first, lo, F in ((True, 2.0 ** -10, 448.0), (False, 2.0 ** -18, 61440.0)):
        codes, s = adamw.encode_state(x, first)
        back = adamw.decode_state(codes, s, first).astype(np.float64)
        each = np.repeat(s, 128)
        # a v below half the least step keeps code 1, a step of 2^-17
        floor = lo if first else 2.0 ** -17
        assert np.all(np.abs(back - x) <= x * (2.0 ** -4 + 2.0 ** -20) + floor * (1 + 2.0 ** -20) * each)
        assert first or np.all(codes[x > 0] >= 1)
        total = np.zeros(1280)
        n = 400
        for seed in range(n):
            c, _ = adamw.encode_state(x, first, seed, 4)
            got = adamw.decode_state(c, s, first).astype(np.float64)
            total += got
            assert np.all(np.abs(got - x) <= x * (2.0 ** -3 + 2.0 ** -20) + 2 * floor * (1 + 2.0 ** -20) * each)
        big = x > 64 * lo * each            # where the least code does not bind
        step = np.maximum(x * 2.0 ** -3, 2 * lo * each)
        # mean of n draws of a variable within one step: six standard deviations of at most step / (2 sqrt n)
        assert np.all(np.abs(total / n - x)[big] <= (6 / (2 * math.sqrt(n)) + 2.0 ** -16) * step[big])
    codes, s = adamw.encode_state(np.array([np.inf] + [1.0] * 200, np.float32), False)
    assert np.isnan(s[0]) and s[1] == np.float32(1 / 61440) and not codes[:128].any() and codes[128] == 0xF7


# ---- refusals of the C entries

def f8(codes=FAKE, ld=128, scales=FAKE, lds=128):
    return _lib.fp8_tensor(codes, ld, scales, lds)


def quant(x=FAKE, rows=64, cols=128, ld=128, fmt=0, kind=0, axis=3, rq="d", cq="d"):
    return _lib.mx_fp8_quantize(x, rows, cols, ld, fmt, kind, axis, f8() if rq == "d" else rq,
                                f8() if cq == "d" else cq, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1), (dict(cols=-8), 1), (dict(fmt=2), 1), (dict(kind=2), 1), (dict(axis=0), 1), (dict(axis=4), 1),
    (dict(x=0), 1), (dict(x=FAKE + 8), 1), (dict(ld=120), 1), (dict(ld=132), 1), (dict(cols=124), 1),
    (dict(rq=None), 1), (dict(cq=None), 1), (dict(rq=f8(codes=0)), 1), (dict(rq=f8(codes=FAKE + 8)), 1),
    (dict(rq=f8(scales=0)), 1), (dict(rq=f8(scales=FAKE + 2)), 1), (dict(rq=f8(ld=112)), 1), (dict(rq=f8(ld=136)), 1),
    (dict(rq=f8(lds=63)), 1), (dict(cq=f8(lds=127)), 1), (dict(cq=f8(ld=64)), 1), (dict(cols=136, ld=136), 1),
    (dict(kind=1, rq=f8(lds=0)), 1), (dict(rows=1 << 40, cols=1 << 20, ld=1 << 20), 1),
    (dict(rows=0), 0), (dict(cols=0), 0),
])
def test_quantize_validation(kw, want):
    assert quant(**kw) == want


def gemm(a="d", af=0, b="d", bf=0, kind=0, M=64, N=64, K=128, c=FAKE, ldc=64, out=0, ws=None, wsb=0):
    return _lib.mx_fp8_gemm(f8() if a == "d" else a, af, f8() if b == "d" else b, bf, kind, M, N, K, c, ldc, out,
                            ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=0), 1), (dict(K=-5), 1), (dict(af=2), 1), (dict(bf=-1), 1),
    (dict(kind=2), 1), (dict(out=2), 1), (dict(a=f8(ld=64)), 1), (dict(K=129), 1), (dict(a=f8(lds=63)), 1),
    (dict(b=f8(lds=63)), 1), (dict(kind=1, b=f8(lds=0)), 1), (dict(a=f8(codes=0)), 1), (dict(b=f8(scales=0)), 1),
    (dict(b=f8(codes=FAKE + 4)), 1), (dict(c=0), 1), (dict(c=FAKE + 2), 1), (dict(c=FAKE + 1, out=1), 1),
    (dict(ldc=63), 1), (dict(ws=FAKE + 8, wsb=64), 1), (dict(wsb=-1), 1), (dict(M=0), 0), (dict(N=0), 0),
])
def test_gemm_validation(kw, want):
    assert gemm(**kw) == want


def step(bits=32, rnd=0, count=1, null=False, tensor=None, **kw):
    p = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    p.update(kw)
    t = dict(w=FAKE, g=FAKE, m=FAKE, v=FAKE, m_scales=FAKE, v_scales=FAKE, copy=FAKE, n=0, grad=0)
    t.update(tensor or {})
    arr = (_lib.AdamwTensorC * 1)(_lib.AdamwTensorC(**t))
    return _lib.mx_adamw_step(None if null else arr, count, bits, _lib.AdamwParamsC(**p), rnd, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(bits=16), 1), (dict(rnd=2), 1), (dict(bits=32, rnd=1), 0), (dict(count=-1), 1), (dict(null=True), 1),
    (dict(beta1=1.0), 1), (dict(beta1=-0.1), 1), (dict(beta2=float("nan")), 1), (dict(eps=-1e-8), 1),
    (dict(eps=float("inf")), 1), (dict(lr=float("nan")), 1), (dict(weight_decay=float("inf")), 1), (dict(step=0), 1),
    (dict(step_dev=FAKE + 4), 1), (dict(lr_dev=FAKE + 2), 1), (dict(grad_scale=FAKE + 1), 1),
    (dict(tensor=dict(n=-1)), 1), (dict(tensor=dict(grad=2)), 1), (dict(tensor=dict(n=8, w=0)), 1),
    (dict(tensor=dict(n=8, g=0)), 1), (dict(tensor=dict(n=8, w=FAKE + 2)), 1), (dict(tensor=dict(n=8, g=FAKE + 2)), 1),
    (dict(tensor=dict(n=8, g=FAKE + 1, grad=1)), 1), (dict(tensor=dict(n=8, m=FAKE + 2)), 1),
    (dict(tensor=dict(n=8, copy=FAKE + 1)), 1), (dict(bits=8, tensor=dict(n=8, m_scales=0)), 1),
    (dict(bits=8, tensor=dict(n=8, v_scales=FAKE + 2)), 1), (dict(tensor=dict(n=1 << 40)), 1),
    (dict(count=0, null=True), 0), (dict(), 0),
])
def test_adamw_validation(kw, want):
    assert step(**kw) == want


def test_adamw_rejects_null_parameters():
    assert _lib.lib().mx_adamw_step(None, 0, 32, None, 0, 0, None) == 1


# ---- refusals of the binding (host tensors: nothing is launched)

def test_quantize_binding_refusals():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    for bad in (dict(x=x[0]), dict(x=x, axis="rows"), dict(x=x, kind="block"), dict(x=x, fmt="e3m4"),
                dict(x=x.t()), dict(x=x[:1].expand(4, 128)),
                dict(x=x, row_out=empty_fp8(4, 256, "cpu")), dict(x=x, row_out=empty_fp8(5, 128, "cpu")),
                dict(x=x, row_out=empty_fp8(4, 128, "cpu", fmt="e5m2")),
                dict(x=x, row_out=empty_fp8(4, 128, "cpu", kind="tile")), dict(x=x)):
        with pytest.raises(ValueError):
            fp8_quantize(**bad)
    with pytest.raises(TypeError):
        fp8_quantize(x.float())


def test_gemm_binding_refusals():
    a, b = empty_fp8(4, 200, "cpu"), empty_fp8(6, 200, "cpu", kind="tile")

    def changed(q, **kw):
        d = dict(codes=q.codes, scales=q.scales, k=q.k, fmt=q.fmt, kind=q.kind)
        d.update(kw)
        return Fp8Tensor(**d)
    for bad in (dict(a=b, b=a), dict(a=a, b=empty_fp8(6, 100, "cpu")), dict(a=changed(a, fmt="x"), b=b),
                dict(a=changed(a, kind="tile"), b=b), dict(a=changed(a, k=300), b=b),
                dict(a=changed(a, codes=a.codes[:, :200]), b=b), dict(a=changed(a, codes=a.codes[:1].expand(4, 256)), b=b),
                dict(a=changed(a, scales=a.scales.t().contiguous()), b=b), dict(a=changed(a, scales=a.scales.double()), b=b),
                dict(a=a, b=changed(b, scales=b.scales[:, :1])), dict(a=a, b=b, out=torch.empty(4, 5)),
                dict(a=a, b=b, out=torch.empty(6, 4).t()), dict(a=a, b=b, out=torch.empty(1, 6).expand(4, 6)),
                dict(a=a, b=b, out_dtype=torch.float16), dict(a=a, b=b)):
        with pytest.raises(ValueError):
            fp8_gemm(**bad)


def test_adamw_binding_refusals():
    w, g = torch.zeros(300), torch.zeros(300)
    s32, s8 = AdamWState.zeros_like(w), AdamWState.zeros_like(w, 8)
    assert s8.m_scale.numel() == 3 and s8.bits == 8 and s32.bits == 32
    with pytest.raises(ValueError):
        AdamWState.zeros_like(w, 16)
    ok = dict(params=[w], grads=[g], states=[s32])
    AdamWTensors(**ok)
    w2 = torch.zeros(300)
    for bad in (dict(params=[w, w2]), dict(grads=[]), dict(grads=[g[:299]]), dict(grads=[g.double()]),
                dict(grads=[torch.zeros(600)[::2]]), dict(params=[w.double()]), dict(params=[torch.zeros(600)[::2]]),
                dict(states=[AdamWState(s8.m, s8.v)]), dict(states=[AdamWState(s8.m, s8.v, s8.m_scale[:2], s8.v_scale)]),
                dict(states=[AdamWState(s32.m, s32.m)]), dict(states=[AdamWState(s32.m, w)]),
                dict(copies=[torch.zeros(300)]), dict(copies=[torch.zeros(299, dtype=torch.bfloat16)]), dict(copies=[]),
                dict(params=[w, w], grads=[g, g], states=[s32, AdamWState.zeros_like(w)]),
                dict(params=[w, w2], grads=[g, g], states=[s32, s32]),
                dict(params=[w, w2], grads=[g, g], states=[s32, AdamWState.zeros_like(w, 8)])):
        with pytest.raises(ValueError):
            AdamWTensors(**{**ok, **bad})
    t = AdamWTensors(**ok)
    for bad in (dict(rounding="up"), dict(lr=torch.zeros(1)[:, None].double()), dict(step=torch.ones(1)),
                dict(step=torch.ones(2, dtype=torch.int64)), dict(grad_scale=2.0), dict(grad_scale=torch.ones(2)), dict()):
        with pytest.raises(ValueError):
            adamw_step(t, **{**dict(lr=1e-3, step=1), **bad})
    adamw_step(AdamWTensors([], [], []), lr=1e-3, step=1)          # nothing to do
    with pytest.raises(_lib.MXError):
        adamw_step(AdamWTensors([], [], []), lr=1e-3, step=0)


def test_operands_of_one_line_and_none():
    for lines, k in ((1, 1), (1, 4096), (0, 128), (3, 5)):
        for kind in ("line", "tile"):
            q = empty_fp8(lines, k, "cpu", kind=kind)
            q.check("q")
            assert q.c_struct().ld_codes >= q.codes.shape[1] and api._fp8_blocks(k) * 128 == q.codes.shape[1]


def test_sizes_past_a_launch_are_refused():
    """A grid holds fewer than 2^32 threads: what would need more is an invalid argument, not a device error."""
    thin = f8(lds=1 << 31)
    assert quant(rows=1 << 30, cols=8, ld=8, rq=thin, cq=f8(ld=1 << 30)) == 1
    assert gemm(M=1, N=1 << 27, a=thin, b=thin, ldc=1 << 27) == 1
    assert gemm(M=1 << 30, N=1, a=thin, b=thin) == 1
    assert gemm(M=1 << 16, N=1 << 21, a=thin, b=thin, ldc=1 << 21) == 1
    assert step(tensor=dict(n=1 << 36)) == 1


def test_shared_memory_is_refused():
    """Operands that a call writes twice: one output for both axes, weights, states or copies that overlap in part."""
    x, q = torch.zeros((128, 128), dtype=torch.bfloat16), empty_fp8(128, 128, "cpu")
    other = empty_fp8(128, 128, "cpu")
    for col in (q, Fp8Tensor(other.codes, q.scales, 128), Fp8Tensor(q.codes, other.scales, 128)):
        with pytest.raises(ValueError, match="share memory"):
            fp8_quantize(x, axis="both", row_out=q, col_out=col)
    none = [empty_fp8(0, 8, "cpu"), empty_fp8(8, 0, "cpu")]        # nothing is written: only the host tensor is refused
    with pytest.raises(ValueError, match="CUDA"):
        fp8_quantize(torch.zeros((0, 8), dtype=torch.bfloat16), axis="both", row_out=none[0], col_out=none[1])
    flat, moments = torch.zeros(1000), torch.zeros(4000)
    m = [moments[1000 * i:1000 * i + 500] for i in range(4)]
    g = torch.zeros(500)
    ok = [AdamWState(m[0], m[1]), AdamWState(m[2], m[3])]
    AdamWTensors([flat[:500], flat[500:]], [g, g], ok)            # one gradient for both is read only
    half = torch.zeros(600, dtype=torch.bfloat16)
    for bad in (dict(params=[flat[:500], flat[499:999]]), dict(states=[AdamWState(moments[:500], moments[100:600]), ok[1]]),
                dict(states=[ok[0], AdamWState(flat[:500], m[3])]), dict(copies=[half[:500], half[100:]]),
                dict(copies=[half[:500], flat[:250].view(torch.bfloat16)])):
        with pytest.raises(ValueError, match="overlaps"):
            AdamWTensors(**{**dict(params=[flat[:500], flat[500:]], grads=[g, g], states=ok), **bad})


def operand_at(buf, at, lines, k, kind="line", pitch=None, scales_at=None, scales=None):
    """An operand whose codes lie in a byte buffer from `at`, and its scales in `scales` (bytes) from `scales_at`."""
    kb = -(-k // 128)
    pitch = pitch or kb * 128
    codes = buf.as_strided((lines, kb * 128), (pitch, 1), at)
    if scales is None:
        return Fp8Tensor(codes, empty_fp8(lines, k, "cpu", kind=kind).scales, k, "e4m3", kind)
    shape = (kb, lines) if kind == "line" else (-(-lines // 128), kb)
    return Fp8Tensor(codes, scales.view(torch.float32).as_strided(shape, (shape[1], 1), scales_at // 4), k, "e4m3", kind)


def test_cast_outputs_that_overlap_in_part_are_refused():
    """Outputs that share some bytes with one another or with x; views side by side in one buffer share none and pass on
    to the next check, which refuses a host tensor."""
    buf = torch.zeros(1 << 17, dtype=torch.uint8)
    x = torch.zeros((128, 128), dtype=torch.bfloat16)
    size = 128 * 128
    other = empty_fp8(128, 128, "cpu")
    xb = buf[:2 * size].view(torch.bfloat16).view(128, 128)
    for bad in (dict(row_out=operand_at(buf, 0, 128, 128), col_out=operand_at(buf, size - 16, 128, 128)),
                dict(row_out=operand_at(buf, 0, 128, 128), col_out=operand_at(buf, 16, 128, 128, pitch=256)),
                dict(row_out=operand_at(buf, 0, 128, 128, pitch=256), col_out=operand_at(buf, 256 * 127, 128, 128, pitch=272)),
                dict(row_out=operand_at(buf, 0, 128, 128), col_out=operand_at(buf, size, 128, 128, scales_at=size - 4, scales=buf)),
                dict(row_out=operand_at(buf, 0, 128, 128, scales_at=256, scales=buf), col_out=other),
                dict(row_out=operand_at(buf, 0, 128, 128, scales_at=size, scales=buf), col_out=operand_at(buf, size + 16, 128, 128)),
                dict(x=xb, row_out=operand_at(buf, 2 * size - 16, 128, 128)),
                dict(x=xb, col_out=operand_at(buf, 2 * size, 128, 128, scales_at=512, scales=buf)),
                dict(x=xb, axis="row", row_out=operand_at(buf, 16, 128, 128))):
        with pytest.raises(ValueError, match="share memory"):
            fp8_quantize(**{**dict(x=x, axis="both"), **bad})
    for good in (dict(row_out=operand_at(buf, 0, 128, 128, pitch=256), col_out=operand_at(buf, 128, 128, 128, pitch=256)),
                 dict(row_out=operand_at(buf, 0, 128, 128), col_out=operand_at(buf, size, 128, 128, scales_at=2 * size, scales=buf)),
                 dict(x=xb, row_out=operand_at(buf, 2 * size, 128, 128), col_out=operand_at(buf, 3 * size, 128, 128)),
                 dict(x=xb, axis="row", row_out=other, col_out=operand_at(buf, 0, 128, 128))):      # col_out is not written
        with pytest.raises(ValueError, match="CUDA"):
            fp8_quantize(**{**dict(x=x, axis="both"), **good})


def test_products_over_their_operands_are_refused():
    buf = torch.zeros(1 << 18, dtype=torch.uint8)
    a, b = operand_at(buf, 0, 20, 128), operand_at(buf, 4096, 24, 128, "tile", scales_at=8192, scales=buf)

    def out(at, dtype, pitch=24):
        return buf.view(dtype).as_strided((20, 24), (pitch, 1), at // dtype.itemsize)
    for c in (out(2560 - 4, torch.float32), out(2560 - 2, torch.bfloat16), out(4096 - 1920 + 4, torch.float32),
              out(4096 + 3068, torch.float32), out(8192, torch.float32), out(8194 - 960, torch.bfloat16),
              out(64, torch.bfloat16, 4000)):
        with pytest.raises(ValueError, match="share memory"):
            fp8_gemm(a, b, out=c)
    # beside the operands: behind a, behind b, and between the rows of an operand of a wide pitch
    wide = operand_at(buf, 16384, 20, 128, pitch=256)
    for q, c in ((a, out(2560, torch.bfloat16)), (a, out(8196, torch.float32)), (wide, out(16384 + 128, torch.float32, 64))):
        with pytest.raises(ValueError, match="CUDA"):
            fp8_gemm(q, b, out=c)


def test_gradients_over_what_a_step_writes_are_refused():
    """A gradient that shares some bytes with a weight, state or copy, of its own tensor or of another, when the list is
    made and when other gradients go in; what they share among themselves is only read."""
    flat, g = torch.zeros(8000), torch.zeros(500)
    w, m = [flat[:500], flat[600:1100]], [flat[1000 * i:1000 * i + 500] for i in range(2, 6)]
    ok = dict(params=w, grads=[g, g], states=[AdamWState(m[0], m[1]), AdamWState(m[2], m[3])],
              copies=[flat[6000:6250].view(torch.bfloat16), None])
    t = AdamWTensors(**ok)
    beside = [flat[500:600], flat[1100:1600], flat[7000:7500]]
    half = flat[:7400].view(torch.bfloat16)
    for bad in (flat[:500], flat[499:999], flat[400:900], flat[101:601], flat[2499:2999], flat[5001:5501], flat[5751:6251],
                half[998:1498], half[12499:12999], half[11600:12100]):
        with pytest.raises(ValueError, match="overlaps"):
            AdamWTensors(**{**ok, "grads": [g, bad]})
        with pytest.raises(ValueError, match="overlaps"):
            t.set_grads([bad, g])
    t.set_grads([beside[1], beside[2]])
    t.set_grads([half[1000:1200].expand(1, 200).reshape(-1).repeat(3)[:500], beside[2]])
    t.set_grads([half[13000:13500], half[12500:13000]])
    assert t.grads[0] is not g
    with pytest.raises(ValueError):
        t.set_grads([g, flat[:500]])
    assert t._c[0].g == t.grads[0].data_ptr() and t._c[1].g == t.grads[1].data_ptr()      # a refused call changes nothing


def test_the_list_of_a_step_cannot_change_under_it():
    """The C entry reads as many tensors as the list was made of, at the addresses they had: the lists cannot grow or be
    replaced, and a state's tensor that its owner replaces lives on, since steps still write it."""
    w, g = torch.zeros(300), torch.zeros(300)
    s = AdamWState.zeros_like(w, 8)
    t = AdamWTensors([w], [g], [s], copies=[torch.zeros(300, dtype=torch.bfloat16)])
    for name in ("params", "grads", "states", "copies"):
        with pytest.raises(AttributeError):
            getattr(t, name).append(w)
        with pytest.raises(AttributeError):
            setattr(t, name, [w, w])
    with pytest.raises(AttributeError):
        t.bits = 32
    old = [weakref.ref(x) for x in (s.m, s.v, s.m_scale, s.v_scale, g, w)]
    s.m, s.v, s.m_scale, s.v_scale = (torch.zeros(1) for _ in range(4))
    del g, w
    gc.collect()
    assert all(r() is not None for r in old)
    assert (t._c[0].m, t._c[0].v_scales) == (old[0]().data_ptr(), old[3]().data_ptr())


def test_workspace_of_any_size_asked_for():
    """Sizes that the product refuses need none, however large: the counts do not wrap."""
    assert _lib.mx_fp8_gemm_workspace(300, 500, 8192, 1) == 16 * 300 * 500 * 4
    top = (1 << 63) - 1
    for M, N, K in (((1 << 42) - 1, (1 << 36) - 1, 4096), (1 << 62, 1 << 62, 1 << 20), (top, top, top), (300, 500, top),
                    (300, 500, (1 << 62) - 1), (-1, 500, 4096), (300, 0, 4096), (300, 500, 0)):
        assert _lib.mx_fp8_gemm_workspace(M, N, K, 0) == _lib.mx_fp8_gemm_workspace(M, N, K, 1) == 0
    assert _lib.mx_fp8_gemm_workspace(300, 500, 8192, 2) == 0


def test_memory_checks_stay_on_the_host():
    """Whatever torch's default device is: a check that made its index tensors there would run on the GPU, and break a
    capture."""
    buf = torch.zeros(1 << 17, dtype=torch.uint8)
    x = torch.zeros((128, 128), dtype=torch.bfloat16)
    row, col = operand_at(buf, 0, 128, 128, pitch=256), operand_at(buf, 128, 128, 128, pitch=256)
    over = operand_at(buf, 112, 128, 128, pitch=256)
    with torch.device("meta"):
        with pytest.raises(ValueError, match="CUDA"):
            fp8_quantize(x, axis="both", row_out=row, col_out=col)
        with pytest.raises(ValueError, match="share memory"):
            fp8_quantize(x, axis="both", row_out=row, col_out=over)
