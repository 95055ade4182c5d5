"""The AdamW step at the ends of its arguments' ranges, and over what outlives a call."""
import pytest

from test_gpu_adamw import check_step, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_smallest_eps(bits):
    """No gradient and no moments: the parameter is left as it is, whatever eps; with some, the formula's step."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32", "bf16"), [3000, 700], seed=20)
    for g in grads:
        g[::3] = 0.0
    before = [p.clone() for p in params]
    opt = mpq.AdamW(params, lr=1e-3, betas=(0.9, 0.99), eps=2.0 ** -126, state_bits=bits, seed=5)
    check_step(opt, grads)
    assert all(torch.equal(p[::3], q[::3]) for p, q in zip(params, before))
    opt.step([torch.zeros_like(g) for g in grads])
    assert all(torch.equal(p[::3], q[::3]) and torch.isfinite(p).all() for p, q in zip(params, before))
    for eps in (1e-39, 2.0 ** -127, 0.0, float("nan")):
        with pytest.raises(ValueError):
            mpq.AdamW(params, eps=eps, state_bits=bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_outlives_a_move(bits):
    """A parameter moves after a step was captured: the eager step that finds it again leaves the graph's plan in place,
    and replays step the parameter where it is now."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32", "bf16"), [3000, 257, 70000], seed=21)
    twin = [p.clone() for p in params]
    a = mpq.AdamW(params, lr=1e-2, state_bits=bits, seed=4)
    b = mpq.AdamW(twin, lr=1e-2, state_bits=bits, seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            a.step(grads, max_norm=1.0)
    torch.cuda.current_stream().wait_stream(side)
    old = params[2]
    params[2] = a.params[2] = old.clone()
    a.step(grads, max_norm=1.0)
    b.step(grads, max_norm=1.0)
    # what a plan that had been let go of would be given to
    others = [torch.full((int(a._table.numel()),), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    left = old.clone()
    for _ in range(3):
        graph.replay()
        b.step(grads, max_norm=1.0)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(params + list(a.state_dict().values()),
                                                     twin + list(b.state_dict().values())))
    assert torch.equal(old, left) and all(bool((o == 255).all()) for o in others)


def test_a_move_is_not_found_while_capturing():
    """The plan is written by the host: refused, with nothing enqueued and nothing changed."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32",), [300], seed=22)
    opt = mpq.AdamW(params, lr=1e-2)
    opt.step(grads)
    opt.params[0] = params[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(ValueError, match="moved"):
                opt.step(grads)
            grads[0].mul_(1.0)   # (a graph of something)
    torch.cuda.current_stream().wait_stream(side)
    check_step(opt, grads)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_resumed_run_rounds_as_the_first(bits, tmp_path):
    """A state_dict carries the seed of the random bits: the steps after it are the same bits, whatever the new seed was."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("bf16", "fp16", "fp32"), [3000, 700, 513], seed=23)
    a = mpq.AdamW(params, state_bits=bits, seed=2 ** 32 - 7)
    a.step(grads)
    twin = [p.clone() for p in params]
    torch.save(a.state_dict(), tmp_path / "state")
    b = mpq.AdamW(twin, state_bits=bits)
    b.load_state_dict(torch.load(tmp_path / "state", weights_only=True))
    assert b.seed == a.seed
    for _ in range(3):
        a.step(grads)
        b.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(params, twin))
    assert all(torch.equal(v, b.state_dict()[k]) for k, v in a.state_dict().items())
    check_step(b, grads)
    old = {k: v for k, v in a.state_dict().items() if k != "seed"}   # (one that was saved without)
    c = mpq.AdamW(twin, state_bits=bits, seed=11)
    c.load_state_dict(old)
    assert c.seed == 11


@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_beyond_float32(bits):
    """The norm is handed back in float32: a step is taken where that is finite, and where it is infinite it is not, although
    every gradient is finite and so is the sum in float64."""
    import torch
    import post_quantization_solver_amd as mpq
    params, grads = problem(("fp32",), [500, 70], seed=24)
    opt = mpq.AdamW(params, state_bits=bits)
    opt.step(grads)
    before = [t.clone() for t in params + list(opt.state_dict().values())]
    large = [g.clone() for g in grads]
    large[0][:4] = 3e38
    for limit in (1.0, float("inf")):
        assert torch.isposinf(opt.step(large, max_norm=limit))
        assert torch.isposinf(opt.step(large, max_norm=limit, grad_scale=-1.0))
        assert all(torch.equal(a, b) for a, b in zip(before, params + list(opt.state_dict().values())))
    # (3e38 twice the square root of 4, halved and more)
    norm = opt.step(large, max_norm=1.0, grad_scale=0.25)
    assert torch.isfinite(norm) and abs(float(norm) / 1.5e38 - 1) < 2.0 ** -22 and int(opt.steps) == 2
    assert all(torch.isfinite(p).all() for p in params)
