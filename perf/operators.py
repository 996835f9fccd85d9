"""Cases of the 8-bit linear-layer operators and the optimizer step, with their plain forms.

Three operators of a linear layer's training step are measured:

  quant  a bf16 matrix cast to E4M3 or E5M2 with a float32 scale for each block of 128 (a line's 128 values, or a
         128 x 128 tile), along its rows, its columns or both;
  gemm   C = A B^T on two such operands, A scaled by lines and B by lines or tiles, to bfloat16 or float32;
  adamw  one AdamW step over a list of float32 weights, states in 32 bits or in 8 (E4M3 first moment, unsigned E5M3
         second moment, a float32 scale for each 128 values), with the bfloat16 copy of the new weights.

The plain forms below are elementary torch operations in float32; exact() computes the same results in float64 from
the definitions, on its own.
"""
import math

import torch

own = False

BLOCK = 128
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126
E5M3_LARGEST = 61440.0           # 1.875 * 2^15: code 0xF7
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.95, 1e-8, 0.1, 3e-4

# Widths of a Llama-3.1-8B block's linears (out, in), q/k/v and gate/up as fused projections.
LINEARS = {"qkv": (6144, 4096), "o": (4096, 4096), "gate_up": (28672, 4096), "down": (4096, 14336)}
BLOCK_WEIGHTS = ",".join(str(o * i) for o, i in LINEARS.values())


def listed():
    return [
        # one token's activation cast before a decode step: latency
        {"name": "quant token", "op": "quant", "rows": 1, "cols": 4096, "kind": "line", "fmt": "e4m3", "axis": "row"},
        # a block's input activation, cast once for Fprop and Wgrad
        {"name": "quant activation", "op": "quant", "rows": 8192, "cols": 4096, "kind": "line", "fmt": "e4m3",
         "axis": "both"},
        # an upstream gradient of the widest linear over a ragged token count, for Dgrad and Wgrad
        {"name": "quant gradient ragged", "op": "quant", "rows": 8001, "cols": 14336, "kind": "line", "fmt": "e5m2",
         "axis": "both"},
        # the gate_up weight, one scale per 128 x 128 tile, for Fprop and Dgrad
        {"name": "quant weight", "op": "quant", "rows": 28672, "cols": 4096, "kind": "tile", "fmt": "e4m3",
         "axis": "both"},
        # one token through the qkv projection: the weight is read once
        {"name": "gemm token", "op": "gemm", "m": 1, "n": 6144, "k": 4096, "kind": "tile", "a": "e4m3", "b": "e4m3",
         "out": "bf16"},
        # a short ragged prompt through the down projection
        {"name": "gemm prompt", "op": "gemm", "m": 333, "n": 4096, "k": 14336, "kind": "tile", "a": "e4m3",
         "b": "e4m3", "out": "bf16"},
        # Fprop of the gate_up projection over a training batch: the largest product
        {"name": "gemm fprop", "op": "gemm", "m": 8192, "n": 28672, "k": 4096, "kind": "tile", "a": "e4m3",
         "b": "e4m3", "out": "bf16"},
        # Wgrad of the down projection over a ragged token count: both operands scaled by lines, E5M2 gradient
        {"name": "gemm wgrad ragged", "op": "gemm", "m": 4096, "n": 14336, "k": 8001, "kind": "line", "a": "e5m2",
         "b": "e4m3", "out": "f32"},
        # the two norm weights of a block: latency
        {"name": "adamw norms", "op": "adamw", "sizes": "4096,4096", "bits": 32, "grad": "bf16", "rounding": "rtne"},
        # a block's linear weights, 32-bit states, the float32 gradients that Wgrad writes
        {"name": "adamw block 32", "op": "adamw", "sizes": BLOCK_WEIGHTS, "bits": 32, "grad": "f32",
         "rounding": "rtne"},
        # the same with 8-bit states and stochastic rounding
        {"name": "adamw block 8", "op": "adamw", "sizes": BLOCK_WEIGHTS, "bits": 8, "grad": "f32", "rounding": "sr"},
        # many tensors of odd sizes (adapters, biases, a small head), bfloat16 gradients
        {"name": "adamw many odd", "op": "adamw", "sizes": ",".join(str(1 + 7919 * i % 300007) for i in range(1, 101)),
         "bits": 8, "grad": "bf16", "rounding": "rtne"},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "adamw"])
    if op == "quant":
        kind = rng.choice(["line", "tile"])
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": 8 * _log(rng, 8, 1792), "kind": kind,
                "fmt": rng.choice(["e4m3", "e5m2"]), "axis": rng.choice(["row", "col", "both"])}
    if op == "gemm":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 14336), "k": _log(rng, 64, 8192),
                "kind": rng.choice(["line", "tile"]), "a": rng.choice(["e4m3", "e5m2"]), "b": "e4m3",
                "out": rng.choice(["bf16", "f32"])}
    count = _log(rng, 1, 40)
    top = _log(rng, 16, 2000000)
    return {"op": op, "sizes": ",".join(str(_log(rng, 1, top)) for _ in range(count)), "bits": rng.choice([8, 32]),
            "grad": rng.choice(["bf16", "f32"]), "rounding": rng.choice(["rtne", "sr"])}


# ---- plain forms ------------------------------------------------------------------------------------------------


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _scales_of(amax, largest):
    """s = max(amax / largest, 2^-126), NaN where the block holds Inf or NaN."""
    s = (amax / largest).clamp_min(TINY)
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, math.nan))


def _cast_lines(x, kind, fmt):
    """Codes (L, padded K) and scales of the lines of a bf16 matrix."""
    lines, k = x.shape
    kb = _padded(k) // BLOCK
    lp = _padded(lines) if kind == "tile" else lines
    v = torch.zeros((lp, kb * BLOCK), dtype=torch.float32, device=x.device)
    v[:lines, :k] = x.to(torch.float32)
    if kind == "line":
        v = v.view(lines, kb, BLOCK)
        s = _scales_of(v.abs().amax(dim=2), LARGEST[fmt])
        each = s.unsqueeze(2)
        scales = s.t().contiguous()
    else:
        v = v.view(lp // BLOCK, BLOCK, kb, BLOCK)
        s = _scales_of(v.abs().amax(dim=(1, 3)), LARGEST[fmt])
        each = s[:, None, :, None]
        scales = s
    y = torch.where(torch.isnan(each), torch.zeros_like(v), v * (1.0 / each))
    return y.reshape(lp, kb * BLOCK)[:lines].to(DTYPE[fmt]), scales


def _quant_plain(s):
    out = {}
    if s["axis"] != "col":
        out["row"] = _cast_lines(s["x"], s["kind"], s["fmt"])
    if s["axis"] != "row":
        out["col"] = _cast_lines(s["x"].t(), s["kind"], s["fmt"])
    return out


def _decoded(codes, scales, kind, fmt):
    """The values an operand stands for: (L, padded K)."""
    lines, kp = codes.shape
    v = codes.view(DTYPE[fmt]).to(torch.float32).view(lines, kp // BLOCK, BLOCK)
    s = scales.t() if kind == "line" else scales.repeat_interleave(BLOCK, dim=0)[:lines]
    return (v * s.unsqueeze(2)).view(lines, kp)


def _gemm_plain(s):
    a = _decoded(s["a_codes"], s["a_scales"], "line", s["a"])
    b = _decoded(s["b_codes"], s["b_scales"], s["kind"], s["b"])
    return torch.mm(a, b.t()).to(OUT[s["out"]])


def _philox(group, stream, seed):
    """16-bit draws of Philox4x32-10, eight for each group: element i of a tensor takes half i % 2 of word (i % 8) // 2
    of the call with counter (i // 8, stream) under key `seed`."""
    low = 0xFFFFFFFF
    c0, c1 = group & low, group >> 32
    c2, c3 = torch.zeros_like(c0) + stream, torch.zeros_like(c0)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), dim=1)
    return torch.stack((words & 0xFFFF, words >> 16), dim=2).view(-1)


def _encode(y, emin, top, r):
    """Codes with 3 mantissa bits of |y|: exponents from emin, saturating at code `top`; r: 16-bit draws, or None."""
    y = y.abs()
    e = torch.where(y > 0, torch.frexp(y).exponent - 1, emin).clamp_min(emin)
    t = torch.ldexp(y, 3 - e)
    c = torch.round(t) if r is None else torch.floor((torch.floor(t * 65536.0) + r) / 65536.0)
    return (c.to(torch.int32) + 8 * (e - emin)).clamp_max(top)


def _e5m3(codes):
    """The values of E5M3 codes: a float16's bits without its sign and its last 7 mantissa bits."""
    seven = torch.full((1,), 7, dtype=torch.int16, device=codes.device)
    return torch.bitwise_left_shift(codes, seven).view(torch.float16)


def _state_values(codes, scales, first):
    v = codes.view(torch.float8_e4m3fn) if first else _e5m3(codes)
    return (v.to(torch.float32).view(-1, BLOCK) * scales.unsqueeze(1)).view(-1)


def _state_codes(v, first, r):
    """8-bit codes and scales of a moment: E4M3 (first) or E5M3 (second, where a value above 0 keeps a code above 0)."""
    b = v.view(-1, BLOCK)
    s = _scales_of(b.abs().amax(dim=1), LARGEST["e4m3"] if first else E5M3_LARGEST)
    bad = torch.isnan(s).unsqueeze(1)
    y = torch.where(bad, torch.zeros_like(b), b * (1.0 / s).unsqueeze(1)).view(-1)
    c = _encode(y, -6, 0x7E, r) if first else _encode(y, -14, 0xF7, r)
    if first:
        c = c + 128 * torch.signbit(y).to(torch.int32)
    else:
        c = torch.where((b > 0) & ~bad, c.view(-1, BLOCK).clamp_min(1), c.view(-1, BLOCK)).view(-1)
    return c.to(torch.uint8), s


def _draws(s, moment):
    """The draws of every place of the flat buffers, each tensor counting from 0 in a stream of its own."""
    if s["rounding"] != "sr":
        return None
    starts = s["starts"]
    group = torch.arange(s["flat"]["w"].numel() // 8, dtype=torch.int64, device=starts.device)
    t = torch.bucketize(8 * group, starts, right=True) - 1
    return _philox(group - starts[t] // 8, 4 + moment + 2 * t, s["seed"] + s["step"])


def _adamw_plain(s):
    """One step on the flat buffers; the places between two tensors hold zeros and keep them."""
    s["step"] += 1
    f = s["flat"]
    c1 = LR / (1.0 - BETA1 ** s["step"])
    c2 = 1.0 / math.sqrt(1.0 - BETA2 ** s["step"])
    g = f["g"].to(torch.float32)
    if s["bits"] == 32:
        m, v = f["m"], f["v"]
    else:
        m, v = _state_values(f["m"], f["m_scale"], True), _state_values(f["v"], f["v_scale"], False)
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * (1.0 - BETA2) * g
    d = torch.sqrt(v) * c2 + EPS
    f["w"].copy_(f["w"] * (1.0 - LR * DECAY) - (m / d) * c1)
    f["copy"].copy_(f["w"])
    if s["bits"] == 8:
        m, m_scale = _state_codes(m, True, _draws(s, 0))
        v, v_scale = _state_codes(v, False, _draws(s, 1))
        f["m_scale"].copy_(m_scale)
        f["v_scale"].copy_(v_scale)
    f["m"].copy_(m)
    f["v"].copy_(v)


# ---- inputs -----------------------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activation(rows, cols, gen):
    """N(0, 1), one column in a thousand 50 times larger."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    hot = torch.rand((1, cols), generator=gen, device="cuda") < 0.001
    return torch.where(hot, 50.0 * x, x).to(torch.bfloat16)


def _gradient(rows, cols, gen):
    """Heavy-tailed values around 1e-3, one in a thousand 100 times larger."""
    u = torch.rand((rows, cols), generator=gen, device="cuda") - 0.5
    g = -1e-3 * torch.sign(u) * torch.log1p(-1.999 * u.abs())
    hot = torch.rand((rows, cols), generator=gen, device="cuda") < 0.001
    return torch.where(hot, 100.0 * g, g).to(torch.bfloat16)


def _weight(rows, cols, gen):
    return (0.02 * torch.randn((rows, cols), generator=gen, device="cuda")).to(torch.bfloat16)


def _optimizer(case, gen):
    """Weights, gradients and moments in flat buffers, as a trainer keeps them, each tensor at a multiple of 128
    elements with zeros up to the next one; the list of the tensors in them; and where the tensors start."""
    sizes = [int(v) for v in case["sizes"].split(",")]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _padded(n))
    total = starts[-1]
    length = torch.tensor([_padded(n) for n in sizes], device="cuda")
    real = torch.arange(total, device="cuda") - torch.tensor(starts[:-1], device="cuda").repeat_interleave(length)
    real = real < torch.tensor(sizes, device="cuda").repeat_interleave(length)

    def normal(size):
        return torch.where(real, size * torch.randn(total, generator=gen, device="cuda"), 0.0)

    flat = {"w": normal(0.02), "g": normal(1e-3)}
    flat["copy"] = flat["w"].to(torch.bfloat16)
    if case["grad"] == "bf16":
        flat["g"] = flat["g"].to(torch.bfloat16)
    flat["m"], flat["v"] = normal(3e-4), torch.where(real, normal(1e-3).square() + 1e-8, 0.0)
    if case["bits"] == 8:
        flat["m"], flat["m_scale"] = _state_codes(flat["m"], True, None)
        flat["v"], flat["v_scale"] = _state_codes(flat["v"], False, None)
    tensors = []
    for at, n in zip(starts, sizes):
        x = {k: flat[k][at:at + n] for k in ("w", "g", "copy", "m", "v")}
        if case["bits"] == 8:
            x |= {k: flat[k][at // BLOCK:(at + _padded(n)) // BLOCK] for k in ("m_scale", "v_scale")}
        tensors.append(x)
    return flat, tensors, torch.tensor(starts[:-1], device="cuda")


def prepare(case, seed):
    gen = _generator(seed)
    s = dict(case)
    if case["op"] == "quant":
        make = _weight if case["kind"] == "tile" else _gradient if case["fmt"] == "e5m2" else _activation
        s["x"] = make(case["rows"], case["cols"], gen)
    elif case["op"] == "gemm":
        make = _gradient if case["a"] == "e5m2" else _activation
        codes, s["a_scales"] = _cast_lines(make(case["m"], case["k"], gen), "line", case["a"])
        s["a_codes"] = codes.view(torch.uint8)
        make = _weight if case["kind"] == "tile" else _activation
        codes, s["b_scales"] = _cast_lines(make(case["n"], case["k"], gen), case["kind"], case["b"])
        s["b_codes"] = codes.view(torch.uint8)
    else:
        s["step"] = 99
        s["seed"] = 7000
        s["flat"], s["tensors"], s["starts"] = _optimizer(case, gen)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------


def _quant_own(s):
    from block_scaled_fp4_hadamard_amd import fp8_quantize
    got = fp8_quantize(s["x"], axis=s["axis"], kind=s["kind"], fmt=s["fmt"])
    return {name: (q.codes.view(DTYPE[s["fmt"]]), q.scales) for name, q in got.items()}


def _gemm_own(s):
    from block_scaled_fp4_hadamard_amd import Fp8Tensor, fp8_gemm
    a = Fp8Tensor(s["a_codes"], s["a_scales"], s["k"], s["a"], "line")
    b = Fp8Tensor(s["b_codes"], s["b_scales"], s["k"], s["b"], s["kind"])
    return fp8_gemm(a, b, out_dtype=OUT[s["out"]])


def _adamw_own(s):
    from block_scaled_fp4_hadamard_amd import AdamWState, AdamWTensors, adamw_step
    if "list" not in s:          # a trainer makes the list of its weights, gradients and states once
        t = s["tensors"]
        s["list"] = AdamWTensors([x["w"] for x in t], [x["g"] for x in t],
                                 [AdamWState(x["m"], x["v"], x.get("m_scale"), x.get("v_scale")) for x in t],
                                 copies=[x["copy"] for x in t])
    s["step"] += 1
    adamw_step(s["list"], lr=LR, step=s["step"], beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
               rounding=s["rounding"], seed=s["seed"] + s["step"])


def run(state):
    s = state
    if s["op"] == "quant":
        return _quant_own(s) if own else _quant_plain(s)
    if s["op"] == "gemm":
        return _gemm_own(s) if own else _gemm_plain(s)
    if own:
        _adamw_own(s)
    else:
        _adamw_plain(s)
    f = s["flat"]
    out = {"w": f["w"], "copy": f["copy"]}
    if s["bits"] == 32:
        out["m"], out["v"] = f["m"], f["v"]
    else:                        # the values that the codes stand for, before the blocks' scales
        out["m"], out["v"] = f["m"].view(torch.float8_e4m3fn), _e5m3(f["v"])
        out["m_scale"], out["v_scale"] = f["m_scale"], f["v_scale"]
    return out


def work(case):
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        outs = 2 if case["axis"] == "both" else 1
        scales = 4.0 * n / BLOCK if case["kind"] == "line" else 4.0 * n / BLOCK ** 2
        return {"bytes": 2 * n + outs * (n + scales), "flops": 2 * n * (1 + outs)}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        b_scales = n * kb if case["kind"] == "line" else -(-n // BLOCK) * kb
        return {"bytes": (m + n) * k + 4 * (m * kb + b_scales) + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * n * k}
    n = sum(int(v) for v in case["sizes"].split(","))
    states = 16.0 if case["bits"] == 32 else 4.0 + 16.0 / BLOCK
    return {"bytes": n * (8 + 2 + (4 if case["grad"] == "f32" else 2) + states), "flops": 15 * n}


# ---- the same in 64 bits ----------------------------------------------------------------------------------------


def _nearest(y, mantissa, emin, largest):
    """The value with `mantissa` bits after the point and exponents from emin that is nearest to y, ties to even."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** (emin - 1)))).clamp_min(emin)
    unit = torch.exp2(e - mantissa)
    return (torch.round(y / unit) * unit).clamp(-largest, largest)


def _drawn(y, emin, largest, r):
    """y rounded up from the level below (3 bits after the point) where its 16-bit fraction and the draw reach 2^16."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** (emin - 1)))).clamp_min(emin)
    unit = torch.exp2(e - 3)
    t = y.abs() / unit
    below = torch.floor(t)
    up = torch.floor((t - below) * 65536.0) + r >= 65536.0
    return torch.where(y < 0, -1.0, 1.0) * ((below + up) * unit).clamp_max(largest)


def _exact_cast(v, kind, fmt):
    """v: float64 (L, K), K and (tiles) L whole blocks."""
    lines, k = v.shape
    top, mantissa, emin = (448.0, 3, -6) if fmt == "e4m3" else (57344.0, 2, -14)
    if kind == "line":
        s = v.abs().reshape(lines, k // 128, 128).max(dim=2).values / top
        each = s.repeat_interleave(128, dim=1)
    else:
        s = v.abs().reshape(lines // 128, 128, k // 128, 128).permute(0, 2, 1, 3).reshape(lines // 128, k // 128, -1)
        s = s.max(dim=2).values / top
        each = s.repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
    y = torch.where(each > 0, v / each.clamp_min(1e-300), torch.zeros_like(v))
    return _nearest(y, mantissa, emin, top), s.t() if kind == "line" else s


def _exact_quant(case, x):
    out = {}
    for name, lines in (("row", x), ("col", x.t())):
        if case["axis"] in (name, "both"):
            n, k = lines.shape
            more = -n % 128 if case["kind"] == "tile" else 0
            v = torch.nn.functional.pad(lines.double(), (0, -k % 128, 0, more))
            codes, s = _exact_cast(v, case["kind"], case["fmt"])
            out[name] = (codes[:n], s)
    return out


def _exact_gemm(s):
    """One block of 128 of K at a time, so that each operand's scales stay apart from the sum they multiply."""
    a, b = s["a_codes"].view(DTYPE[s["a"]]), s["b_codes"].view(DTYPE[s["b"]])
    m, n = a.shape[0], b.shape[0]
    c = torch.zeros((m, n), dtype=torch.float64, device=a.device)
    line = torch.arange(n, device=a.device)
    for at in range(0, a.shape[1], 4096):
        x = a[:, at:at + 4096].double()
        y = b[:, at:at + 4096].double()
        for j in range(0, x.shape[1], 128):
            block = (at + j) // 128
            x[:, j:j + 128] *= s["a_scales"][block].double()[:, None]
            sb = s["b_scales"][block] if s["kind"] == "line" else s["b_scales"][:, block][line // 128]
            y[:, j:j + 128] *= sb.double()[:, None]
        c += x @ y.t()
    return c


def _exact_adamw(s):
    step = s["step"] + 1
    flat = {k: [] for k in ("w", "copy", "m", "v") + (() if s["bits"] == 32 else ("m_scale", "v_scale"))}
    for t, x in enumerate(s["tensors"]):
        n = x["w"].numel()
        g, w = x["g"].double(), x["w"].double()
        if s["bits"] == 32:
            m, v = x["m"].double(), x["v"].double()
        else:
            m = x["m"].view(torch.float8_e4m3fn).double() * x["m_scale"].double().repeat_interleave(128)[:n]
            v = (x["v"].to(torch.int16) * 128).view(torch.float16).double()
            v = v * x["v_scale"].double().repeat_interleave(128)[:n]
        m = BETA1 * m + (1.0 - BETA1) * g
        v = BETA2 * v + (1.0 - BETA2) * g * g
        mean, var = m / (1.0 - BETA1 ** step), v / (1.0 - BETA2 ** step)
        w = w - LR * DECAY * w - LR * mean / (var.sqrt() + EPS)
        new = {"w": w, "copy": w, "m": m, "v": v}
        if s["bits"] == 8:
            for name, top, emin, stream in (("m", 448.0, -6, 4 + 2 * t), ("v", 61440.0, -14, 5 + 2 * t)):
                z = torch.nn.functional.pad(new[name], (0, -n % 128)).view(-1, 128)
                scale = (z.abs().max(dim=1, keepdim=True).values / top).clamp_min(TINY)
                z = (z / scale).view(-1)[:n]
                if s["rounding"] == "sr":
                    group = torch.arange(-(-n // 8), device=z.device)
                    q = _drawn(z, emin, top, _philox(group, stream, s["seed"] + step)[:n])
                else:
                    q = _nearest(z, 3, emin, top)
                if name == "v":
                    q = torch.where(z > 0, q.clamp_min(2.0 ** -17), q)
                new[name], new[name + "_scale"] = q, scale.view(-1)
        for k in flat:
            more = 0 if k.endswith("_scale") else -n % 128
            flat[k].append(torch.nn.functional.pad(new[k], (0, more)))
    return {k: torch.cat(v) for k, v in flat.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(case, s["x"])
    return _exact_gemm(s) if case["op"] == "gemm" else _exact_adamw(s)
