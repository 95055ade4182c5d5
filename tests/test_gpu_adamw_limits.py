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
