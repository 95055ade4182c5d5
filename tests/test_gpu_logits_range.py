"""Distillation and log probabilities at the ends of their range, against float64:
students whose unlisted mass is far below what float32 holds about the row's
maximum, and more rows than one launch has workgroups.

Tolerances as in test_gpu_logits.py.  Where the unlisted tokens lie G nats below
the listed ones, their log mass is G's product with log2(e) as a float32, half
a step of 2^-23 off at most: 2^-24 / 1.44 G, doubled for the maximum that it is
taken from, so that the loss carries 2^-23 G times the teacher's remainder beside
2^-17 of the weight."""
import numpy as np
import pytest

from oracle import ops_oracle as R
from parity_helpers import dev, host
from test_gpu_logits import STEP, rows, teacher_list

pytestmark = pytest.mark.gpu


def far_tail(g, t, V, k, dtype, gaps):
    """Rows of k listed tokens around 0 and unlisted ones `gap` below, and a teacher with a remainder."""
    import torch
    z = rows(g, t, V, dtype, spread=2.0).clone()
    ids = np.stack([g.permutation(V)[:k] for _ in range(t)]).astype(np.int32)
    hidden = torch.ones(t, V, dtype=torch.bool, device="cuda").scatter_(1, dev(ids).long(), False)
    down = torch.from_numpy(np.resize(np.array(gaps, np.float32), t)).cuda()[:, None]
    low = torch.clamp_min(z.float() - down, torch.finfo(z.dtype).min)
    z = torch.where(hidden, low.to(z.dtype), z)
    lp = np.log(g.dirichlet(np.ones(k), t) * 0.75).astype(np.float32)   # a quarter outside the list
    return z, ids, lp


GAPS = [30.0, 44.0, 60.0, 90.0, 95.0, 103.0, 130.0, 1e3, 1e4, 6e4]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,V,k", [(10, 1000, 64), (10, 40003, 5), (10, 70001, 128), (130, 4099, 20), (130, 40003, 1)])
def test_distill_far_tail(dtype, t, V, k):
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(V + k)
    z, ids, lp = far_tail(g, t, V, k, dtype, GAPS)
    weights = (0.5 + g.random(t)).astype(np.float32)
    loss, grad, scale = R.distill(z.double().cpu().numpy(), ids, lp.astype(np.float64), 1.0, True, weights)
    r = mpq.distill(z, dev(ids), dev(lp), tail=True, weights=dev(weights))
    torch.cuda.synchronize()
    assert np.isfinite(loss).all() and np.isfinite(grad).all()
    got = host(r["loss"]).astype(np.float64)
    # (the loss is at least the remainder times the gap: 2^-23 of it covers the gap's part)
    assert (np.abs(got - loss) <= 2.0 ** -22 * np.abs(loss) + 2.0 ** -17 * weights).all(), np.abs(got / loss - 1).max()
    tol = STEP[dtype] * np.abs(grad) + 2.0 ** -16 * scale + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    err = np.abs(r["grad"].double().cpu().numpy() - grad)
    assert (err <= tol).all(), (err / tol).max()
    zc = z.clone()
    over = mpq.distill(zc, dev(ids), dev(lp), tail=True, weights=dev(weights), grad=zc)
    assert torch.equal(over["grad"], r["grad"]) and torch.equal(over["loss"], r["loss"])
    assert torch.equal(mpq.distill(z, dev(ids), dev(lp), tail=True, weights=dev(weights), grad=False)["loss"], r["loss"])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t", [6, 132])
def test_distill_masked_unlisted(dtype, t):
    """Unlisted tokens masked by the type's lowest value, by -inf but for some far ones, and by -inf alone: there the
    loss is infinite and the gradient the listed tokens' alone."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(t)
    V, k = 20003, 7
    z, ids, lp = far_tail(g, t, V, k, dtype, [0.0])
    hidden = torch.ones(t, V, dtype=torch.bool, device="cuda").scatter_(1, dev(ids).long(), False)
    kind = torch.arange(t, device="cuda")[:, None] % 3
    far = torch.arange(V, device="cuda")[None, :] % 1000 == 3
    low = torch.finfo(z.dtype).min
    z = torch.where(hidden & (kind == 0), low, z)
    z = torch.where(hidden & (kind == 1), torch.where(far, -300.0, float("-inf")).to(z.dtype), z)
    z = torch.where(hidden & (kind == 2), float("-inf"), z)
    loss, grad, scale = R.distill(z.double().cpu().numpy(), ids, lp.astype(np.float64), 1.0, True)
    r = mpq.distill(z, dev(ids), dev(lp), tail=True)
    got = host(r["loss"]).astype(np.float64)
    endless = np.arange(t) % 3 == 2
    assert np.isposinf(loss[endless]).all() and np.isposinf(got[endless]).all()
    fin = ~endless
    assert (np.abs(got[fin] - loss[fin]) <= 2.0 ** -22 * np.abs(loss[fin]) + 2.0 ** -17).all()
    tol = STEP[dtype] * np.abs(grad) + 2.0 ** -16 * scale + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    assert (np.abs(r["grad"].double().cpu().numpy() - grad) <= tol).all()
