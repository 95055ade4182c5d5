"""The AdamW step over many tensors against float64, step by step from the state
that the library itself holds.

Tolerances.  32-bit moments: the gradient's factor, the rate 1 - beta, beta, their
products and the sum are a rounding of 2^-24 each, two more for the square:
2^-22 of the magnitudes added for m, 2^-21 for v.  The parameter: two roundings of
its own size (2^-23 |p|), and the update, whose m is off by 2^-22 of its
magnitudes and whose corrections, root, product and quotient round some eight
times: 2^-20 of the magnitudes' update.  16-bit parameters are rounded to either
neighbour: a whole step more, 2 eps / 2 = 2^-7 or 2^-10 of the value (float16: and 2^-24
below its normal range, to the nearest).  Codes of 8 bits are computed in float64
on both sides, in the same order (scales half way between two floats are not
rare: with decimal betas a largest element is a multiple of 1 / 150 of a float's
step), and an element is within 2^-50 of a border only by a chance of some 2^-40:
they have to be equal, and so do their scales.
"""
import ctypes

import numpy as np
import pytest

from oracle import ops_oracle as R

pytestmark = pytest.mark.gpu

SIZES = [1, 255, 256, 257, 2047, 2048, 2049, 4096, 0, 5000, 33]


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def problem(dtypes, sizes, seed, shift=0):
    """Parameters (from an odd address on, with shift) and gradients of sizes that differ by orders of magnitude."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    params, grads = [], []
    for k, n in enumerate(sizes):
        dt = dtype_of(dtypes[k % len(dtypes)])
        kind = 10.0 ** (k % 5 - 3)
        for out, size in ((params, 1.0), (grads, kind)):
            buf = torch.zeros(n + shift + 8, dtype=dt, device="cuda")
            buf[shift:shift + n] = (torch.randn(n, generator=g, device="cuda") * size *
                                    torch.exp(torch.randn(n, generator=g, device="cuda"))).to(dt)
            out.append(buf[shift:shift + n])
    return params, grads


def f64(t):
    return t.detach().double().cpu().numpy()


def expected_norm(grads, grad_scale):
    return np.sqrt(sum(float((f64(g) ** 2).sum()) for g in grads)) * grad_scale


def check_step(opt, grads, grad_scale=1.0, max_norm=None, lr_factor=None, factor_value=1.0):
    """One step against the formulas, from the state that is there."""
    import torch
    torch.cuda.synchronize()
    before = [f64(p) for p in opt.params]
    old = {k: v.cpu().numpy().copy() for k, v in opt.state_dict().items()}
    t = int(old["step"][0]) + 1
    norm = opt.step(grads, grad_scale=grad_scale, max_norm=max_norm, lr_factor=lr_factor)
    torch.cuda.synchronize()
    new = {k: v.cpu().numpy() for k, v in opt.state_dict().items()}
    assert int(new["step"][0]) == t
    factor = grad_scale
    if max_norm is not None:
        n = expected_norm(grads, grad_scale)
        assert abs(float(norm) - n) <= 2.0 ** -23 * n
        factor = grad_scale * min(1.0, max_norm / n) if n > 0 else grad_scale
    else:
        assert norm is None
    factor = float(np.float32(factor))
    for k, (p, g) in enumerate(zip(opt.params, grads)):
        n, at = p.numel(), opt.offsets[k]
        if n == 0:
            continue
        pad = -n % 256
        whole = slice(at, at + n + pad)
        gp = np.pad(f64(g), (0, pad))
        if opt.state_bits == 8:
            blocks = slice(at // 256, (at + n + pad) // 256)
            m0 = R.decode8(old["m"][whole], old["m_scale"][blocks], 3)
            v0 = R.decode8(old["r"][whole], old["r_scale"][blocks], 4) ** 2
        else:
            m0, v0 = old["m"][whole].astype(np.float64), old["v"][whole].astype(np.float64)
        lr, decay = opt._rates[0][k] * factor_value, opt._rates[1][k]
        want, m, v, size = R.adamw(np.pad(before[k], (0, pad)), gp, m0, v0, t, lr, opt.betas, opt.eps, decay, factor)
        if opt.state_bits == 8:
            h = R.adamw_words(opt.seed, t, at, n + pad).astype(np.int64)
            for name, val, F, bits in (("m", m, 3, h & 0xffff), ("r", np.sqrt(v), 4, h >> 16)):
                code, scale = R.encode8(val, F, bits)
                assert np.array_equal(new[name + "_scale"][blocks], scale), (k, name)
                assert np.array_equal(new[name][whole], code), (k, name, (new[name][whole] != code).sum())
        else:
            grads_m = opt.betas[0] * np.abs(m0) + (1 - opt.betas[0]) * np.abs(gp * factor)
            assert (np.abs(new["m"][whole] - m) <= 2.0 ** -22 * grads_m + 1e-40).all(), k
            assert (np.abs(new["v"][whole] - v) <= 2.0 ** -21 * v + 1e-40).all(), k
        want, size, got = want[:n], size[:n], f64(p)
        tol = 2.0 ** -23 * np.abs(before[k]) + 2.0 ** -20 * size
        if p.dtype != torch.float32:
            step = 2.0 ** -7 if p.dtype == torch.bfloat16 else 2.0 ** -10
            tol = tol + step * np.abs(want) + (2.0 ** -24 if p.dtype == torch.float16 else 0.0)
        assert (np.abs(got - want) <= tol + 1e-40).all(), (k, (np.abs(got - want) / (tol + 1e-40)).max())
    return norm


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtypes", [("fp32",), ("bf16",), ("fp16",), ("fp32", "bf16", "fp16")])
@pytest.mark.parametrize("shift", [0, 1])
def test_steps(bits, dtypes, shift):
    import post_quantization_solver_amd as mpq
    params, grads = problem(dtypes, SIZES, seed=bits + shift, shift=shift)
    opt = mpq.AdamW(params, lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.05, state_bits=bits, seed=1234567)
    for _ in range(3):
        check_step(opt, grads)
    _, more = problem(dtypes, SIZES, seed=99, shift=shift)
    n = expected_norm(more, 0.25)
    check_step(opt, more, grad_scale=0.25, max_norm=0.3 * n)
    check_step(opt, more, grad_scale=0.25, max_norm=4.0 * n, lr_factor=0.5, factor_value=0.5)
    for t in params + grads:   # what lies about the tensors is left alone
        whole = t.untyped_storage()
        buf = t.new_empty(0).set_(whole, 0, (whole.nbytes() // t.element_size(),))
        assert not buf[:shift].any() and not buf[shift + t.numel():].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [1, 440, 441, 900])
def test_many_tensors(bits, count):
    """More than one launch's tensors; a rate and a decay each."""
    import post_quantization_solver_amd as mpq
    sizes = [SIZES[k % len(SIZES)] if k % 7 == 0 else 1 + k % 300 for k in range(count)]
    params, grads = problem(("fp32", "bf16"), sizes, seed=count)
    opt = mpq.AdamW(params, lr=[1e-3 * (1 + k % 3) for k in range(count)], weight_decay=[0.1 * (k % 2) for k in range(count)],
                    state_bits=bits, seed=count)
    check_step(opt, grads)
    check_step(opt, grads, max_norm=0.5 * expected_norm(grads, 1.0))


@pytest.mark.parametrize("bits", [32, 8])
def test_large(bits):
    """Units that go round the grid, uneven moments, several launches' worth of workgroups."""
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32", "bf16"), [5_000_001, 777_777], seed=3)
    opt = mpq.AdamW(params, lr=1e-2, state_bits=bits, seed=2 ** 32 - 1)
    for _ in range(2):
        check_step(opt, grads, max_norm=0.7 * expected_norm(grads, 1.0))


@pytest.mark.parametrize("bits", [32, 8])
def test_extremes(bits):
    """Zeros, float32's largest and smallest magnitudes, beta 0."""
    import torch
    import post_quantization_solver_amd as mpq
    g = torch.zeros(2048, device="cuda")
    g[256:512] = 1e-40
    g[512:768] = 1e18
    g[768:1024] = torch.logspace(-30, 15, 256, device="cuda")
    g[1030] = -5.0
    g[1280:1536] = 1e-20
    g[1536] = 1e-3
    for betas in ((0.9, 0.999), (0.0, 0.5), (0.5, 0.0)):
        p = torch.ones(2048, device="cuda")
        opt = mpq.AdamW([p], lr=0.1, betas=betas, eps=1e-6, state_bits=bits)
        for k in range(3):
            check_step(opt, [g if k != 1 else torch.zeros_like(g)])
        m, v = opt.moments()
        assert torch.isfinite(m).all() and torch.isfinite(v).all() and torch.isfinite(p).all()


def test_moments():
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32",), SIZES, seed=5)
    opt = mpq.AdamW(params, state_bits=8, seed=9)
    opt.step(grads)
    m, v = opt.moments()
    s = {k: t.cpu().numpy() for k, t in opt.state_dict().items()}
    want_m, want_r = R.decode8(s["m"], s["m_scale"], 3), R.decode8(s["r"], s["r_scale"], 4)
    assert np.array_equal(m.cpu().numpy(), want_m.astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), (want_r ** 2).astype(np.float32))
    # every code
    both = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)
    opt.m[:256], opt.r[:256] = both, both
    opt.m_scale[0], opt.r_scale[0] = 0.37, 3.1e-5
    m, v = (t[:256].cpu().numpy() for t in opt.moments())
    code, one = np.arange(256, dtype=np.uint8), np.ones(1, np.float32)
    assert np.array_equal(m, R.decode8(code, np.float32(0.37) * one, 3).astype(np.float32))
    assert np.array_equal(v, (R.decode8(code, np.float32(3.1e-5) * one, 4) ** 2).astype(np.float32))


def test_increments_below_a_step_are_kept():
    """A second moment that grows by a thousandth a step, far under a code's: its mean over many elements grows with it.

    65536 elements, all but the blocks' largest with the same gradients: each one's v is right on average, its own
    deviation (the codes' squares are a tenth apart, and a step's rounding is as uncertain as the step is long)
    below 0.4 of it, that of the mean of 65280 below 0.4 / 255: five of them, 2^-7."""
    import torch
    import post_quantization_solver_amd as mpq
    n = 65536
    p = torch.zeros(n, device="cuda")
    opt = mpq.AdamW([p], lr=0.0, betas=(0.9, 0.999), state_bits=8, seed=7)
    g0 = torch.full((n,), 0.1, device="cuda")
    g0[::256] = 30.0   # the block's largest, and much larger than the others
    v = np.zeros(n)
    for t in range(120):
        opt.step([g0])
        v = 0.999 * v + 0.001 * f64(g0) ** 2
    got = f64(opt.moments()[1])
    rest = np.arange(n) % 256 != 0
    ratio = got[rest] / v[rest]
    assert abs(ratio.mean() - 1) < 2.0 ** -7, ratio.mean()
    assert ratio.std() < 0.4


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_that_are_not_taken(bits):
    """A gradient that is not finite, with the norm asked for: nothing changes; without: its element's (its block's) state."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32", "bf16"), [700, 1500], seed=6)
    opt = mpq.AdamW(params, state_bits=bits, seed=1)
    opt.step(grads)
    before = [t.clone() for t in params] + [t.clone() for t in opt.state_dict().values()]
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = [t.clone() for t in grads]
        g[1][1499] = bad
        for limit in (1.0, float("inf")):
            norm = opt.step(g, max_norm=limit)
            assert not torch.isfinite(norm)
            assert all(torch.equal(a, b) for a, b in zip(before, params + list(opt.state_dict().values())))
    check_step(opt, grads, max_norm=float("inf"))
    g = [t.clone() for t in grads]
    g[0][300] = float("nan")
    opt.step(g)
    m, v = opt.moments()
    spoilt = slice(300, 301) if bits == 32 else slice(256, 512)
    for t in (m, v):
        bad = torch.isnan(t)
        assert bad[spoilt].all() and int(bad.sum()) == spoilt.stop - spoilt.start
    assert torch.isnan(params[0][300]) and int(torch.isnan(params[0]).sum()) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_captured(bits):
    """Replays count their own steps and follow a device learning rate; eager work between them."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32", "fp16"), [3000, 257, 70000], seed=8)
    twin = [p.clone() for p in params]
    rate = torch.ones((), device="cuda")
    a = mpq.AdamW(params, lr=1e-2, state_bits=bits, seed=4)
    b = mpq.AdamW(twin, lr=1e-2, state_bits=bits, seed=4)
    a.step(grads, max_norm=1.0, lr_factor=rate)
    b.step(grads, max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            norm = a.step(grads, max_norm=1.0, lr_factor=rate)
    torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        rate.fill_(0.5 ** k)
        for g in grads:
            g.mul_(-0.7)
        graph.replay()
        want = b.step(grads, max_norm=1.0, lr_factor=0.5 ** k)
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        assert all(torch.equal(x, y) for x, y in zip(params + list(a.state_dict().values()),
                                                     twin + list(b.state_dict().values())))
        (grads[0] * 2).sum().item()
    check_step(a, grads)


def test_other_stream_and_same_bits():
    """On another stream than the current one, twice the same bits; another seed, others."""
    import torch
    import post_quantization_solver_amd as mpq
    runs = []
    for seed, other in ((1, False), (1, True), (2, False)):
        params, grads = problem(("bf16", "fp32"), [100_001, 4096], seed=10)
        opt = mpq.AdamW(params, state_bits=8, seed=seed)
        stream = torch.cuda.Stream() if other else torch.cuda.current_stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for _ in range(3):
                opt.step(grads, max_norm=1.0)
        torch.cuda.synchronize()
        runs.append(params + list(opt.state_dict().values()))
    assert all(torch.equal(a, b) for a, b in zip(runs[0], runs[1]))
    assert not torch.equal(runs[0][0], runs[2][0])


def test_state_is_carried_over_and_moved_parameters_are_found():
    import torch
    import post_quantization_solver_amd as mpq
    for bits in (8, 32):
        params, grads = problem(("fp32",), [500, 3000], seed=12)
        a = mpq.AdamW(params, state_bits=bits, seed=3)
        a.step(grads)
        twin = [p.clone() for p in params]
        b = mpq.AdamW(twin, state_bits=bits, seed=3)
        b.load_state_dict({k: v.clone() for k, v in a.state_dict().items()})
        params[1].data = params[1].clone()   # another address
        a.step(grads)
        b.step(grads)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(params, twin))
        with pytest.raises(ValueError):
            b.load_state_dict({"step": a.steps})
        wrong = a.state_dict()
        wrong["m"] = wrong["m"][:256]
        with pytest.raises(ValueError):
            b.load_state_dict(wrong)


def test_refusals():
    import torch
    import post_quantization_solver_amd as mpq
    p = torch.zeros(10, device="cuda")
    for bad in ([], [p.cpu()], [p.double()], [torch.zeros(4, 4, device="cuda")[:, 1]]):
        with pytest.raises((ValueError, TypeError)):
            mpq.AdamW(bad)
    for kw in (dict(state_bits=16), dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)), dict(eps=0.0), dict(lr=[1.0, 2.0])):
        with pytest.raises(ValueError):
            mpq.AdamW([p], **kw)
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(weight_decay=-0.1)):
        with pytest.raises(mpq.MPQError):
            mpq.AdamW([p], **kw)
    with pytest.raises(mpq.MPQError):   # the same parameter twice, and one that overlaps another
        mpq.AdamW([p, p])
    with pytest.raises(mpq.MPQError):
        mpq.AdamW([p[:6], p[5:]])
    opt = mpq.AdamW([p], state_bits=32)
    g = torch.zeros(10, device="cuda")
    for bad in ([], [g, g], [g.cpu()], [g.half()], [g[:9]], [torch.zeros(20, device="cuda")[::2]], [None]):
        with pytest.raises((ValueError, TypeError)):
            opt.step(bad)
    for limit in (0.0, -1.0, float("nan")):
        with pytest.raises(ValueError):
            opt.step([g], max_norm=limit)
    for kw in (dict(grad_scale=float("inf")), dict(lr_factor=-1.0)):
        with pytest.raises(mpq.MPQError):
            opt.step([g], **kw)
    with pytest.raises(ValueError):
        opt.step([g], lr_factor=torch.ones(2, device="cuda"))
    assert int(opt.steps) == 0 and not p.any()


def test_far_places():
    """Moments whose places are beyond 32 bits (the C entry: two tensors far apart)."""
    import torch
    import post_quantization_solver_amd as mpq
    from post_quantization_solver_amd import binding as B
    lib = mpq.load_library()
    at, n = (1 << 32) + 512, 1000
    elements = at + 1024
    p, g = torch.ones(n, device="cuda"), torch.randn(n, device="cuda")
    m, r = (torch.zeros(elements, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, rs = (torch.zeros(elements // 256, device="cuda") for _ in range(2))
    steps = torch.zeros(1, dtype=torch.int32, device="cuda")
    tensors = (B.AdamWTensor * 1)(B.AdamWTensor(p.data_ptr(), n, at, 0.1, 0.0, 2, 0))
    nb = lib.mpq_adamw_plan_bytes(tensors, 1)
    table, plan = torch.empty(nb, dtype=torch.uint8, device="cuda"), B.AdamWPlan()
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.mpq_adamw_plan(tensors, 1, table.data_ptr(), nb, stream, ctypes.byref(plan)) == 0
    assert plan.elements == elements
    state = B.AdamWState(steps.data_ptr(), m.data_ptr(), r.data_ptr(), ms.data_ptr(), rs.data_ptr(), elements, 8, 77)
    opts = B.AdamWOptions(0.9, 0.99, 1e-8, 1.0, 0.0, 1.0, None, None)
    rc = lib.mpq_adamw(ctypes.byref(plan), (ctypes.c_void_p * 1)(g.data_ptr()), ctypes.byref(opts), ctypes.byref(state), stream)
    torch.cuda.synchronize()
    assert rc == 0 and int(steps) == 1
    gp = np.pad(f64(g), (0, 24))
    h = R.adamw_words(77, 1, at, 1024).astype(np.int64)
    _, m1, v1, _ = R.adamw(np.zeros(1024), gp, np.zeros(1024), np.zeros(1024), 1, 0.1, (0.9, 0.99), 1e-8, 0.0, 1.0)
    for codes, scales, val, F, bits in ((m, ms, m1, 3, h & 0xffff), (r, rs, np.sqrt(v1), 4, h >> 16)):
        code, scale = R.encode8(val, F, bits)
        assert np.array_equal(codes[at:].cpu().numpy(), code) and np.array_equal(scales[at // 256:].cpu().numpy(), scale)
    assert not m[:at].any() and not r[:at].any()
