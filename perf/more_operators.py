"""Cases of a block's norms and of the optimizer that orthogonalizes its updates, with their plain forms.

Four operators of a transformer block's training step are measured:

  norm       layer norm of the rows of a bf16 or float32 matrix, or its RMS form (no mean, no bias): y and the
             statistics that the backward pass takes;
  norm_grad  its backward pass: the input's gradient and, summed over the rows, the weight's and the bias's;
  ortho      the nearest semi-orthogonal matrix of each gradient of a list, roughly, by five Newton-Schulz steps
             X <- a X + (b A + c A A) X, A = X X^T, from X = G / (|G| + eps), to bfloat16;
  muon       one optimizer step over a list of float32 weight matrices: momentum, its orthogonalized update, decoupled
             weight decay, and the bfloat16 copy of the new weights.

The plain forms below are elementary torch operations in float32; exact() computes the same results in float64 from
the definitions, on its own.
"""
import math

import torch

own = False

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
NORM_EPS = 1e-5
STEPS, A, B, C, ORTHO_EPS = 5, 3.4445, -4.7750, 2.0315, 1e-7
MOMENTUM, DECAY, LR = 0.95, 0.1, 5e-5          # the learning rate of a schedule's last part

# Weights (out, in) of a Llama-3.1-8B block's linears, q/k/v and gate/up as fused projections.
BLOCK_SHAPES = "6144x4096,4096x4096,28672x4096,4096x14336"


def listed():
    return [
        # one token's hidden state before a decode step: latency
        {"name": "norm token", "op": "norm", "rows": 1, "cols": 4096, "type": "bf16", "weight": "bf16", "kind": "layer"},
        # a training batch's hidden states before a block's first linear
        {"name": "norm activation", "op": "norm", "rows": 8192, "cols": 4096, "type": "bf16", "weight": "bf16",
         "kind": "layer"},
        # per-head norm of a batch's queries: 8192 tokens of 32 heads of 128
        {"name": "norm heads", "op": "norm", "rows": 262144, "cols": 128, "type": "bf16", "weight": "f32",
         "kind": "rms"},
        # float32 activations of an odd width over a ragged token count
        {"name": "norm odd", "op": "norm", "rows": 2001, "cols": 5003, "type": "f32", "weight": "f32",
         "kind": "layer"},
        # the backward pass of a short sequence: few rows, so that the weight's sum is short as well
        {"name": "norm grad short", "op": "norm_grad", "rows": 33, "cols": 4096, "type": "bf16", "weight": "f32",
         "kind": "rms"},
        # the backward pass over a training batch's hidden states
        {"name": "norm grad activation", "op": "norm_grad", "rows": 8192, "cols": 4096, "type": "bf16",
         "weight": "bf16", "kind": "layer"},
        # an inner norm of an odd width over a ragged token count, float32
        {"name": "norm grad odd", "op": "norm_grad", "rows": 4001, "cols": 14335, "type": "f32", "weight": "f32",
         "kind": "layer"},
        # a small model's projection: latency
        {"name": "ortho small", "op": "ortho", "shapes": "128x256", "grad": "bf16"},
        # the output projection's gradient
        {"name": "ortho square", "op": "ortho", "shapes": "4096x4096", "grad": "f32"},
        # tall and wide matrices of odd sizes, orthogonalized together
        {"name": "ortho odd", "op": "ortho", "shapes": "1403x777,999x2047,2500x1001,333x3999", "grad": "f32"},
        # the projections of four small blocks: many matrices that fill the chip only together
        {"name": "muon small blocks", "op": "muon", "shapes": ",".join(["768x512,512x512,2816x512,512x1408"] * 4),
         "grad": "bf16"},
        # all linears of a Llama-3.1-8B block: the largest
        {"name": "muon block", "op": "muon", "shapes": BLOCK_SHAPES, "grad": "f32"},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "ortho", "muon"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 32, 16384)
        rows = min(_log(rng, 1, 65536), 50_000_000 // cols)
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "f32"]),
                "weight": rng.choice(["bf16", "f32"]), "kind": rng.choice(["layer", "rms"])}
    count = _log(rng, 1, 8)
    top = _log(rng, 64, 8192 if count == 1 else 2048)
    shapes = []
    for _ in range(count):
        rows, cols = _log(rng, 16, top), _log(rng, 16, top)
        shapes.append("%dx%d" % (rows, cols))
    return {"op": op, "shapes": ",".join(shapes), "grad": rng.choice(["bf16", "f32"])}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


# ---- plain forms ------------------------------------------------------------------------------------------------


def _norm_plain(s):
    x = s["x"].to(torch.float32)
    mean = x.mean(dim=1) if s["kind"] == "layer" else None
    d = x if mean is None else x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(dim=1) + NORM_EPS)
    y = d * rstd[:, None] * s["weight"].to(torch.float32)
    if mean is not None:
        y = y + s["bias"].to(torch.float32)
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_grad_plain(s):
    layer = s["kind"] == "layer"
    x, dy = s["x"].to(torch.float32), s["dy"].to(torch.float32)
    h = (x - s["mean"][:, None] if layer else x) * s["rstd"][:, None]
    g = dy * s["weight"].to(torch.float32)
    dx = g - h * (g * h).mean(dim=1, keepdim=True)
    if layer:
        dx = dx - g.mean(dim=1, keepdim=True)
    dx = (dx * s["rstd"][:, None]).to(s["x"].dtype)
    return {"dx": dx, "dweight": (dy * h).sum(dim=0), "dbias": dy.sum(dim=0) if layer else None}


def _ortho_plain(u):
    """Five Newton-Schulz steps in float32 on the orientation with fewer rows than columns."""
    tall = u.shape[0] > u.shape[1]
    x = u.to(torch.float32)
    x = x / (torch.sqrt((x * x).sum()) + ORTHO_EPS)
    x = x.t().contiguous() if tall else x
    for _ in range(STEPS):
        a = torch.mm(x, x.t())
        x = A * x + torch.mm(B * a + C * torch.mm(a, a), x)
    return x.t() if tall else x


def _muon_one(t):
    """One matrix's step, in place."""
    g = t["g"].to(torch.float32)
    t["m"].copy_(t["m"] * MOMENTUM + g * (1.0 - MOMENTUM))
    o = _ortho_plain(g * (1.0 - MOMENTUM) + t["m"] * MOMENTUM)
    t["w"].copy_(t["w"] * (1.0 - LR * DECAY) - o * (LR * 0.2 * math.sqrt(max(g.shape))))
    t["copy"].copy_(t["w"])


# ---- inputs -----------------------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activation(rows, cols, gen):
    """N(0, 1) around a little offset for each row, one column in a thousand 50 times larger."""
    x = torch.randn((rows, cols), generator=gen, device="cuda") + 0.2 * torch.randn((rows, 1), generator=gen, device="cuda")
    hot = torch.rand((1, cols), generator=gen, device="cuda") < 0.001
    return torch.where(hot, 50.0 * x, x)


def _gradient(rows, cols, gen):
    """Heavy-tailed values around 1e-3, one in a thousand 100 times larger."""
    u = torch.rand((rows, cols), generator=gen, device="cuda") - 0.5
    g = -1e-3 * torch.sign(u) * torch.log1p(-1.999 * u.abs())
    hot = torch.rand((rows, cols), generator=gen, device="cuda") < 0.001
    return torch.where(hot, 100.0 * g, g)


def _weight_gradient(rows, cols, gen):
    """What a linear's Wgrad gives: a few strong directions of falling size, over the noise of the others."""
    rank = max(1, min(rows, cols, 64) // 2)
    fall = torch.arange(1, rank + 1, device="cuda", dtype=torch.float32).reciprocal()
    left = torch.randn((rows, rank), generator=gen, device="cuda") * fall
    strong = torch.mm(left, torch.randn((rank, cols), generator=gen, device="cuda"))
    return 1e-3 * (strong + 0.1 * torch.randn((rows, cols), generator=gen, device="cuda"))


def prepare(case, seed):
    gen = _generator(seed)
    s = dict(case)
    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activation(rows, cols, gen).to(TYPE[case["type"]])
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(TYPE[case["weight"]])
        s["bias"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(TYPE[case["weight"]])
        if case["op"] == "norm_grad":
            s["dy"] = _gradient(rows, cols, gen).to(TYPE[case["type"]])
            forward = _norm_plain(s)
            s["mean"], s["rstd"] = forward["mean"], forward["rstd"]
        return s
    s["tensors"] = []
    for rows, cols in _shapes(case):
        t = {"g": _weight_gradient(rows, cols, gen).to(TYPE[case["grad"]])}
        if case["op"] == "muon":
            t["w"] = 0.02 * torch.randn((rows, cols), generator=gen, device="cuda")
            t["m"] = t["g"].to(torch.float32) + _weight_gradient(rows, cols, gen)
            t["copy"] = t["w"].to(torch.bfloat16)
        s["tensors"].append(t)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------


def _norm_own(s):
    from block_scaled_fp4_hadamard_amd import layer_norm
    y, mean, rstd = layer_norm(s["x"], s["weight"], s["bias"] if s["kind"] == "layer" else None, eps=NORM_EPS,
                               kind=s["kind"])
    return {"y": y, "mean": mean, "rstd": rstd}


def _norm_grad_own(s):
    from block_scaled_fp4_hadamard_amd import layer_norm_grad
    dx, dweight, dbias = layer_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], kind=s["kind"])
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


def _ortho_own(s):
    from block_scaled_fp4_hadamard_amd import orthogonalize
    return orthogonalize([t["g"] for t in s["tensors"]], steps=STEPS, coefficients=(A, B, C), eps=ORTHO_EPS,
                         out_dtype=torch.bfloat16)


def _muon_own(s):
    from block_scaled_fp4_hadamard_amd import MuonTensors, muon_step
    if "list" not in s:          # a trainer makes the list of its weights, gradients and momenta once
        t = s["tensors"]
        s["list"] = MuonTensors([x["w"] for x in t], [x["g"] for x in t], [x["m"] for x in t],
                                copies=[x["copy"] for x in t])
    muon_step(s["list"], lr=LR, momentum=MOMENTUM, weight_decay=DECAY, steps=STEPS, coefficients=(A, B, C),
              eps=ORTHO_EPS, adjust="rms")


def run(state):
    s = state
    if s["op"] == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if s["op"] == "norm_grad":
        return _norm_grad_own(s) if own else _norm_grad_plain(s)
    if s["op"] == "ortho":
        return _ortho_own(s) if own else [_ortho_plain(t["g"]).to(torch.bfloat16) for t in s["tensors"]]
    if own:
        _muon_own(s)
    else:
        [_muon_one(t) for t in s["tensors"]]
    return [{k: t[k] for k in ("w", "m", "copy")} for t in s["tensors"]]


def work(case):
    if case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        size, weight = (2 if case["type"] == "bf16" else 4), (2 if case["weight"] == "bf16" else 4)
        layer = case["kind"] == "layer"
        stats = 4 * rows * (2 if layer else 1)
        if case["op"] == "norm":
            return {"bytes": 2 * size * rows * cols + weight * cols * (2 if layer else 1) + stats,
                    "flops": 8 * rows * cols}
        return {"bytes": 3 * size * rows * cols + (weight + 4 * (2 if layer else 1)) * cols + stats,
                "flops": 15 * rows * cols}
    size = 2 if case["grad"] == "bf16" else 4
    total = {"bytes": 0, "flops": 0}
    for rows, cols in _shapes(case):
        m, n = min(rows, cols), max(rows, cols)
        # the two symmetric products count once for each pair of their elements
        total["flops"] += STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)
        total["bytes"] += m * n * (size + (2 if case["op"] == "ortho" else 8 + 8 + 2))
    return total


# ---- the same in 64 bits ----------------------------------------------------------------------------------------


def _exact_norm(case, s):
    x, w = s["x"].double(), s["weight"].double()
    if case["kind"] == "rms":
        rstd = 1.0 / (x.pow(2).sum(dim=1) / case["cols"] + NORM_EPS).sqrt()
        return {"y": x * rstd.unsqueeze(1) * w, "mean": None, "rstd": rstd}
    mean = x.sum(dim=1) / case["cols"]
    var = (x - mean.unsqueeze(1)).pow(2).sum(dim=1) / case["cols"]
    rstd = 1.0 / (var + NORM_EPS).sqrt()
    return {"y": (x - mean.unsqueeze(1)) * rstd.unsqueeze(1) * w + s["bias"].double(), "mean": mean, "rstd": rstd}


def _exact_norm_grad(case, s):
    """From y_i = w_i h_i + b_i, h = (x - mean) rstd: dL/dx = rstd (g - P g), P the projection on what the statistics fix."""
    n = case["cols"]
    dy, r = s["dy"].double(), s["rstd"].double().unsqueeze(1)
    h = s["x"].double() * r
    g = dy * s["weight"].double()
    if case["kind"] == "layer":
        h = h - s["mean"].double().unsqueeze(1) * r
        inner = g - g.sum(dim=1, keepdim=True) / n - h * ((g * h).sum(dim=1, keepdim=True) / n)
    else:
        inner = g - h * ((g * h).sum(dim=1, keepdim=True) / n)
    return {"dx": r * inner, "dweight": torch.einsum("rc,rc->c", dy, h),
            "dbias": dy.sum(dim=0) if case["kind"] == "layer" else None}


def _exact_ortho(u):
    """Each step in float64, the smaller Gram matrix on its own side of X."""
    x = u / (torch.linalg.vector_norm(u) + ORTHO_EPS)
    for _ in range(STEPS):
        if x.shape[0] <= x.shape[1]:
            g = x @ x.t().contiguous()
            x = A * x + (B * g + C * (g @ g)) @ x
        else:
            g = x.t().contiguous() @ x
            x = A * x + x @ (B * g + C * (g @ g))
    return x


def _exact_muon(t):
    g, m, w = t["g"].double(), t["m"].double(), t["w"].double()
    m = MOMENTUM * m + (1.0 - MOMENTUM) * g
    o = _exact_ortho(MOMENTUM * m + (1.0 - MOMENTUM) * g)
    w = w - LR * (DECAY * w + 0.2 * math.sqrt(max(w.shape)) * o)
    return {"w": w, "m": m, "copy": w}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "norm_grad":
        return _exact_norm_grad(case, s)
    if case["op"] == "ortho":
        return [_exact_ortho(t["g"].double()) for t in s["tensors"]]
    return [_exact_muon(t) for t in s["tensors"]]
