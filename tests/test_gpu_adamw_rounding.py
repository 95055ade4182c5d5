"""How 16-bit parameters are rounded, bit by bit against the stated hash.

The value before rounding is known to 2^-23 |p| + 2^-20 of the update (test_gpu_adamw.py), some 2^-14 of a step of
float16 and 2^-16 of bfloat16: an element has to be what the random word makes of some value in that interval, which for
all but one in a thousand is one value (either neighbour would pass for a quarter to a half of them otherwise).
"""
import numpy as np
import pytest

from oracle import ops_oracle as R
from test_gpu_adamw import f64, problem

pytestmark = pytest.mark.gpu


def rounded(v, drop, u):
    """|v| (float64, at least 2^-13) to 24 - drop bits, up where the word's low bits u say."""
    bits = np.abs(v).astype(np.float32).view(np.int32).astype(np.int64)
    return np.sign(v) * ((bits + (u & ((1 << drop) - 1))) & -(1 << drop)).astype(np.int32).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,drop", [("bf16", 16), ("fp16", 13)])
@pytest.mark.parametrize("shift", [0, 1])
def test_words(bits, dtype, drop, shift):
    import post_quantization_solver_amd as mpq
    params, grads = problem((dtype,), [40_000, 257, 30_001], seed=30, shift=shift)
    lr, betas, eps, decay, seed = 3e-3, (0.9, 0.99), 1e-8, 0.05, 99
    opt = mpq.AdamW(params, lr=lr, betas=betas, eps=eps, weight_decay=decay, state_bits=bits, seed=seed)
    for t in (1, 2, 3):
        m, v = (f64(s) for s in opt.moments())
        old = [f64(p) for p in params]
        opt.step(grads)
        for p, p0, g, at in zip(params, old, grads, opt.offsets):
            n = len(p0)
            # (moments of 8 bits stand for float64 products that moments() rounds: 2^-23 of the update's terms)
            want, _, _, size = R.adamw(p0, f64(g), m[at:at + n], v[at:at + n], t, lr, betas, eps, decay, 1.0)
            tol = 2.0 ** -23 * np.abs(p0) + 2.0 ** -19 * size
            keep = np.abs(want) > 2.0 ** -13 + tol
            u = R.mix(R.adamw_words(seed, t, at, n) ^ np.uint64(0x9E3779B9)).astype(np.int64)
            lo = rounded(np.sign(want) * (np.abs(want) - tol), drop, u)[keep]
            hi = rounded(np.sign(want) * (np.abs(want) + tol), drop, u)[keep]
            got = f64(p)[keep]
            assert (np.abs(lo) <= np.abs(got)).all() and (np.abs(got) <= np.abs(hi)).all()
            assert (np.sign(got) == np.sign(want[keep])).all()
            if n > 1000:
                assert (lo != hi).mean() < 2.0 ** -9
                nearest = rounded(want, drop, np.full(n, 1 << (drop - 1)))[keep]
                assert ((got != nearest).mean() > 0.1) and ((got != rounded(want, drop, 0 * u)[keep]).mean() > 0.1)


@pytest.mark.parametrize("dtype,step", [("bf16", 2.0 ** -8), ("fp16", 2.0 ** -11)])
def test_updates_below_a_step_are_kept(dtype, step):
    """Updates of a sixteenth of a step (below 1), 32 of them: the mean moves by all of it.

    A step's rounding has a variance of step^2 / 16 at most, 32 of them 2 step^2: the mean of 65536 is off by
    1.42 step / 256, five times that 0.028 step, where all that is moved is two steps; the updates themselves are good
    to 2^-19 of their size."""
    import torch
    import post_quantization_solver_amd as mpq
    n = 65536
    p = torch.full((n,), 0.99, device="cuda").to(dict(bf16=torch.bfloat16, fp16=torch.float16)[dtype])
    start = float(p[0])
    opt = mpq.AdamW([p], lr=step / 16, betas=(0.9, 0.999), state_bits=32, seed=7)
    g = torch.ones_like(p)
    for _ in range(32):
        opt.step([g])
    assert abs(float(p.double().mean()) - (start - 2 * step)) < 0.03 * step
    assert len(p.unique()) > 3
