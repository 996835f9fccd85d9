"""GPU parity of the AdamW step against the oracle: weights, bf16 copies, moments, 8-bit codes and scales bit for bit."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_hadamard_amd import AdamWState, AdamWTensors, adamw_step, fp8_gemm, fp8_quantize, synth
from gpu_helpers import announce, assert_bytes_equal
from oracle import adamw, fp8
from test_fp8_gpu import tolerance

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def draw(sizes, bits, rng, zero=False):
    """Host weights, and moments as the oracle holds them."""
    out = []
    for n in sizes:
        w = (0.02 * rng.standard_normal(n)).astype(np.float32)
        m = (1e-3 * rng.standard_normal(n)).astype(np.float32) * (not zero)
        v = ((1e-3 * rng.standard_normal(n)) ** 2).astype(np.float32) * (not zero)
        s = (m, v) if bits == 32 else adamw.encode_state(m, True) + adamw.encode_state(v, False)
        out.append([w, s])
    return out


def gradient(n, rng, bf16):
    g = (1e-3 * rng.laplace(size=n) * np.where(rng.random(n) < 0.01, 100.0, 1.0)).astype(np.float32)
    if n > 300:
        g[n // 2:n // 2 + 128] = 0.0
    return fp8.bf16_values(synth.f32_to_bf16_bits(g)) if bf16 else g


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def state_of(s, bits):
    return AdamWState(cuda(s[0]), cuda(s[1])) if bits == 32 else AdamWState(cuda(s[0]), cuda(s[2]), cuda(s[1]), cuda(s[3]))


def grads_of(gs, bf16):
    return [cuda(g).bfloat16() if bf16 else cuda(g) for g in gs]


def oracle_step(host, gs, bits, c, scale=None, seed=None):
    for t, (h, g) in enumerate(zip(host, gs)):
        if bits == 32:
            w, m, v = adamw.update(h[0], g, *h[1], c, scale)
            h[0], h[1] = w, (m, v)
        else:
            h[0], h[1] = adamw.step8(h[0], g, h[1], c, scale, seed, t)


def compare(tensors, host, bits, what):
    for t, (w, s, copy, h) in enumerate(zip(tensors.params, tensors.states, tensors.copies, host)):
        name = "%s tensor %d " % (what, t)
        assert_bytes_equal(w.cpu().numpy().view(np.uint32), h[0].view(np.uint32), name + "w")
        if copy is not None:
            assert_bytes_equal(copy.view(torch.int16).cpu().numpy().view(np.uint16), synth.f32_to_bf16_bits(h[0]), name + "copy")
        got = [s.m, s.v] if bits == 32 else [s.m, s.m_scale, s.v, s.v_scale]
        for part, x, y in zip(("m", "v") if bits == 32 else ("m", "m_scale", "v", "v_scale"), got, h[1]):
            x = x.cpu().numpy()
            if x.dtype == np.float32:
                assert np.array_equal(np.isnan(x), np.isnan(y)), name + part
                x, y = np.nan_to_num(x).view(np.uint32), np.nan_to_num(y).view(np.uint32)
            assert_bytes_equal(x, y, name + part)


CASES = [(32, "rtne", False), (32, "sr", True), (8, "rtne", False), (8, "rtne", True), (8, "sr", False), (8, "sr", True)]


@pytest.mark.parametrize("bits,rounding,bf16", CASES)
@pytest.mark.parametrize("sizes", [(1,), (7, 8, 9), (127, 128, 129, 0, 1), (2047, 2048, 2049, 5000), (100003,)])
def test_steps_match_the_oracle(sizes, bits, rounding, bf16):
    rng = np.random.default_rng(sum(sizes) + bits)
    host = draw(sizes, bits, rng, zero=True)
    tensors = AdamWTensors([cuda(h[0]) for h in host], [cuda(h[0]) for h in host], [state_of(h[1], bits) for h in host],
                           copies=[torch.zeros(n, dtype=torch.bfloat16, device="cuda") if t % 2 == 0 else None
                                   for t, n in enumerate(sizes)])
    for step in range(1, 5):
        announce("adamw %s %d %s %s step %d" % (sizes, bits, rounding, bf16, step))
        gs = [gradient(n, rng, bf16) for n in sizes]
        tensors.set_grads(grads_of(gs, bf16))
        scale = None if step % 2 else 0.37
        adamw_step(tensors, step=step, rounding=rounding, seed=77 + step, **HYPER,
                   grad_scale=None if scale is None else torch.full((1,), scale, device="cuda"))
        torch.cuda.synchronize()
        oracle_step(host, gs, bits, adamw.coefficients(step=step, **HYPER), scale, 77 + step if rounding == "sr" else None)
        compare(tensors, host, bits, "step %d" % step)


@pytest.mark.parametrize("bits,rounding", [(32, "rtne"), (8, "sr")])
def test_many_tensors(bits, rounding):
    """More tensors than one launch takes, empty ones among them, and both gradient types in one list."""
    rng = np.random.default_rng(11)
    sizes = [int(v) for v in rng.integers(0, 4000, 131)]
    sizes[3] = sizes[48] = sizes[130] = 0
    host = draw(sizes, bits, rng)
    gs = [gradient(n, rng, t % 3 == 0) for t, n in enumerate(sizes)]
    tensors = AdamWTensors([cuda(h[0]) for h in host], [cuda(g).bfloat16() if t % 3 == 0 else cuda(g) for t, g in enumerate(gs)],
                           [state_of(h[1], bits) for h in host],
                           copies=[torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes])
    announce("adamw many %d" % bits)
    adamw_step(tensors, step=9, rounding=rounding, seed=5, **HYPER)
    torch.cuda.synchronize()
    oracle_step(host, gs, bits, adamw.coefficients(step=9, **HYPER), None, 5 if rounding == "sr" else None)
    compare(tensors, host, bits, "many")


@pytest.mark.parametrize("bits", [32, 8])
def test_any_alignment(bits):
    """Tensors that start at every element of larger buffers: the results are the same, the elements around untouched."""
    rng = np.random.default_rng(12)
    n = 1000
    for off in (1, 2, 3, 4, 8):
        host = draw([n], bits, rng)
        g = gradient(n, rng, True)

        def at(x, dtype, off=off):
            buf = torch.full((x.size + 32,), 3, dtype=dtype, device="cuda")
            view = buf[off:off + x.size]
            view.copy_(cuda(x))
            return buf, view
        parts = [at(host[0][0], torch.float32), at(g, torch.bfloat16), at(np.zeros(n, np.float32), torch.bfloat16)]
        state = torch.float32 if bits == 32 else torch.uint8
        parts += [at(x, state if x.size == n else torch.float32) for x in host[0][1]]
        views = [v for _, v in parts]
        s = AdamWState(*views[3:]) if bits == 32 else AdamWState(views[3], views[5], views[4], views[6])
        announce("adamw offset %d bits %d" % (off, bits))
        t = AdamWTensors([views[0]], [views[1]], [s], copies=[views[2]])
        adamw_step(t, step=3, **HYPER)
        torch.cuda.synchronize()
        oracle_step(host, [g], bits, adamw.coefficients(step=3, **HYPER))
        compare(t, host, bits, "offset %d" % off)
        for buf, v in parts:
            v.fill_(3)
            assert bool((buf == 3).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_edge_values(bits):
    """Inf and NaN gradients, gradients whose squares underflow or overflow, eps 0 over zero moments, beta 0."""
    rng = np.random.default_rng(13)
    n = 128 * 12 + 5
    for hyper in (HYPER, dict(HYPER, eps=0.0), dict(HYPER, beta1=0.0, beta2=0.0), dict(HYPER, weight_decay=0.0, lr=0.0)):
        host = draw([n], bits, rng, zero=True)
        g = gradient(n, rng, False)
        g[5], g[130], g[300] = np.inf, np.nan, -np.inf
        g[384:512] *= np.float32(1e-25)
        g[512:640] *= np.float32(1e24)
        g[640:768] = 0.0
        g[768:896] = np.float32(1e-42)
        announce("adamw edge bits %d %s" % (bits, hyper))
        t = AdamWTensors([cuda(host[0][0])], [cuda(g)], [state_of(host[0][1], bits)])
        adamw_step(t, step=1, **hyper)
        torch.cuda.synchronize()
        oracle_step(host, [g], bits, adamw.coefficients(step=1, **hyper))
        w = t.params[0].cpu().numpy()
        assert np.array_equal(np.isnan(w), np.isnan(host[0][0]))
        t.params[0].copy_(cuda(np.nan_to_num(w)))
        host[0][0] = np.nan_to_num(host[0][0])
        compare(t, host, bits, "edge")


def test_device_step_and_rate():
    """step and lr read on the device give the host's numbers to the bit, through a captured graph whose replays move both
    on, with eager work between the replays."""
    rng = np.random.default_rng(14)
    for bits in (32, 8):
        host = draw([3000, 77], bits, rng)
        gs = [gradient(n, rng, False) for n in (3000, 77)]
        tensors = AdamWTensors([cuda(h[0]) for h in host], grads_of(gs, False), [state_of(h[1], bits) for h in host])
        step = torch.tensor([40], dtype=torch.int64, device="cuda")
        lr = torch.tensor([1e-3], device="cuda")
        hyper = dict(HYPER, lr=lr)
        announce("adamw device step bits %d" % bits)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            adamw_step(tensors, step=step, **hyper)
        for k in range(3):
            g.replay()
            torch.cuda.synchronize()
            c = adamw.coefficients(step=40 + 3 * k, **dict(HYPER, lr=float(np.float32(1e-3 * (1 - 0.25 * k)))))
            oracle_step(host, gs, bits, c)
            compare(tensors, host, bits, "replay %d" % k)
            step += 3
            lr.fill_(1e-3 * (1 - 0.25 * (k + 1)))
    big = torch.tensor([2 ** 31 + 5], dtype=torch.int64, device="cuda")      # the bias corrections have reached 1
    adamw_step(tensors, step=big, **HYPER)
    torch.cuda.synchronize()
    oracle_step(host, gs, 8, adamw.coefficients(step=2 ** 31 + 5, **HYPER))
    compare(tensors, host, 8, "late")


def test_linear_layer_training_steps():
    """Two training steps of one linear in 8 bits, as the operators are used together: cast X, W (tiles) and dY, Fprop,
    Dgrad and Wgrad, AdamW with 8-bit states on the float32 master weight, whose bf16 copy the next step casts.  Every
    result against the oracle running the same steps on its own operands; the AdamW step takes the GPU's dW on both
    sides, so that its codes must agree bit for bit."""
    rng = np.random.default_rng(15)
    T, O, I = 200, 264, 392
    w = (0.02 * rng.standard_normal((O, I))).astype(np.float32)
    master, copy = cuda(w), cuda(w).bfloat16()
    dw = torch.empty((O, I), device="cuda")
    opt = AdamWTensors([master], [dw], [AdamWState.zeros_like(master, bits=8)], copies=[copy])
    host = [[w.reshape(-1), (np.zeros(O * I, np.uint8), np.zeros(-(-O * I // 128), np.float32)) * 2]]

    def close(got, pair, a_fmt, kind, bf16):
        (a, b) = pair
        c, g = fp8.gemm_ref(a, a_fmt, b, "e4m3", kind)
        assert np.all(np.abs(got.float().cpu().numpy() - c) <= tolerance(c, g, a[0].shape[1] // 128, bf16))
    for step in (1, 2):
        xb = synth.activation(T, I, rng)
        gb = synth.gradient(T, O, rng)
        x, dy = (torch.from_numpy(v.view(np.int16)).cuda().view(torch.bfloat16) for v in (xb, gb))
        announce("fp8 linear step %d" % step)
        qx = fp8_quantize(x, axis="both")
        qw = fp8_quantize(copy, axis="both", kind="tile")
        qd = fp8_quantize(dy, axis="both", fmt="e5m2")
        y = fp8_gemm(qx["row"], qw["row"], out_dtype=torch.bfloat16)
        dx = fp8_gemm(qd["row"], qw["col"], out_dtype=torch.bfloat16)
        fp8_gemm(qd["col"], qx["col"], out=dw)
        adamw_step(opt, step=step, rounding="sr", seed=100 + step, **HYPER)
        torch.cuda.synchronize()
        wb = synth.f32_to_bf16_bits(host[0][0].reshape(O, I))
        rx, rw, rd = (fp8.quantize_ref(b, "both", k, f) for b, k, f in ((xb, "line", "e4m3"), (wb, "tile", "e4m3"), (gb, "line", "e5m2")))
        close(y, (rx["row"], rw["row"]), "e4m3", "tile", True)
        close(dx, (rd["row"], rw["col"]), "e5m2", "tile", True)
        close(dw, (rd["col"], rx["col"]), "e5m2", "line", False)
        oracle_step(host, [dw.cpu().numpy().reshape(-1)], 8, adamw.coefficients(step=step, **HYPER), None, 100 + step)
        assert_bytes_equal(master.cpu().numpy().reshape(-1).view(np.uint32), host[0][0].view(np.uint32), "master")
        assert_bytes_equal(copy.view(torch.int16).cpu().numpy().view(np.uint16), synth.f32_to_bf16_bits(host[0][0]).reshape(O, I), "copy")
        assert_bytes_equal(opt.states[0].v.cpu().numpy().reshape(-1), host[0][1][2], "v codes")


def test_stochastic_rounding_draws_anew_at_every_replay():
    """A captured 8-bit step with its step on the device: replay t takes the draws of key seed + t, which are those of an
    eager call with that seed, so that a moment whose gradients stand still keeps moving.  Eager work between replays."""
    rng = np.random.default_rng(18)
    sizes = (1000, 5, 4097)
    host = draw(sizes, 8, rng)
    gs = [gradient(n, rng, False) for n in sizes]
    tensors = AdamWTensors([cuda(h[0]) for h in host], grads_of(gs, False), [state_of(h[1], 8) for h in host])
    eager = AdamWTensors([cuda(h[0]) for h in host], grads_of(gs, False), [state_of(h[1], 8) for h in host])
    step = torch.tensor([6], dtype=torch.int64, device="cuda")
    seed = 2 ** 64 - 9                      # the key passes 2^64 within the replays
    announce("adamw sr graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        adamw_step(tensors, step=step, rounding="sr", seed=seed, **HYPER)
    for t in range(6, 11):
        g.replay()
        torch.cuda.synchronize()
        oracle_step(host, gs, 8, adamw.coefficients(step=t, **HYPER), None, (seed + t) % 2 ** 64)
        compare(tensors, host, 8, "replay %d" % t)
        adamw_step(eager, step=t, rounding="sr", seed=(seed + t) % 2 ** 64, **HYPER)
        compare(eager, host, 8, "eager %d" % t)
        step += 1


def test_second_moment_moves_in_a_graph():
    """1 - beta2 of 2^-12 moves v by less than half a code step of 2^-4 at each step: round-to-nearest would keep every
    code, and so would draws that repeat.  v starts at 1/4 of g^2; after n steps its exact value is g^2 (1 - 3/4 beta2^n),
    and the mean over the elements follows it: one step's rounding is unbiased (16-bit draws: to 2^-16 of a step) and off
    by less than a code step, at most 2^-3 of v <= g^2, so the mean of N elements after n steps is within
    6 sqrt(n / N) 2^-3 / 2 (six standard deviations, each draw's at most half a step) + n 2^-19 of g^2, and float32 adds
    four roundings a step, n 2^-22."""
    N, n, beta2 = 128 * 512, 400, 1.0 - 2.0 ** -12
    w, g = torch.zeros(N, device="cuda"), torch.full((N,), 1e-3, device="cuda")
    # the last of each block sets the scale: its gradient is twice the others', its v the square of it all along
    g[127::128] = 2e-3
    v = (g * g).cpu().numpy() * np.where(np.arange(N) % 128 == 127, 1.0, 0.25).astype(np.float32)
    vc, vs = adamw.encode_state(v, False)
    start = adamw.decode_state(vc, vs, False)
    state = AdamWState(torch.zeros(N, dtype=torch.uint8, device="cuda"), cuda(vc), torch.zeros(N // 128, device="cuda"), cuda(vs))
    tensors = AdamWTensors([w], [g], [state])
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    announce("adamw sr drift")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        adamw_step(tensors, lr=0.0, step=step, beta2=beta2, rounding="sr", seed=3)
        step += 1
    for _ in range(n):
        graph.replay()
    torch.cuda.synchronize()
    got = adamw.decode_state(state.v.cpu().numpy(), state.v_scale.cpu().numpy(), False).astype(np.float64)
    small = np.arange(N) % 128 != 127
    gg = float(np.float32(1e-3)) ** 2
    want = gg + (start[small].astype(np.float64).mean() - gg) * beta2 ** n
    bound = (6 * np.sqrt(n / small.sum()) * 2.0 ** -4 + n * 2.0 ** -19 + n * 2.0 ** -22) * gg
    print("mean v / g^2: %.5f, exact %.5f, bound %.5f" % (got[small].mean() / gg, want / gg, bound / gg))
    assert abs(got[small].mean() - want) <= bound


@pytest.mark.parametrize("bits", [32, 8])
def test_autograd_notices_what_the_operators_write(bits):
    """A backward whose forward saved a weight, a copy, a moment, or an output that a later call has written raises instead
    of using the new values; tensors that the call only reads still give gradients."""
    w = torch.nn.Parameter(torch.randn(256, 256, device="cuda"))
    g, copy = torch.randn(256, 256, device="cuda"), torch.zeros(256, 256, dtype=torch.bfloat16, device="cuda")
    state = AdamWState.zeros_like(w, bits)
    other = torch.ones(256, 256, device="cuda", requires_grad=True)
    tensors = AdamWTensors([w], [g], [state], copies=[copy])
    held = [(other * w.detach()).sum(), (other * copy).sum(), (other * (state.m if bits == 32 else state.v_scale[0])).sum()]
    read = (other * g).sum()
    announce("adamw autograd %d" % bits)
    adamw_step(tensors, lr=1e-3, step=1)
    for y in held:
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    read.backward()
    assert torch.equal(other.grad, g)
    q = fp8_quantize(copy, axis="both")
    c = torch.zeros(256, 256, device="cuda")
    held = [(other * c).sum(), (other * q["row"].scales[0]).sum(), (other * q["col"].scales[0]).sum()]
    read = (other * copy).sum()
    fp8_quantize(copy, axis="row", row_out=q["row"])
    fp8_gemm(q["row"], q["row"], out=c)
    for y in held[:2]:
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    held[2].backward()                      # the column output was not written
    read.backward()
