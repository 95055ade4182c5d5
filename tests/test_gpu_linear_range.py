"""A packed layer's gradients at the ends of their range, against float64."""
import numpy as np
import pytest

from oracle import ops_oracle as R
from parity_helpers import dev
from test_gpu_linear import STEP, dtype_of, f64, make_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name,group", [("e865536", 0), ("s16", 0), ("s16", 64), ("s16", 50)])
def test_backward_of_vanishing_gradients(dtype, name, group):
    """Tokens whose gradient is about 1e-35, beside zeros, under scales of 8 and more, next to an ordinary token.
    dx's tolerance as in test_gpu_linear.py: the sums (m / 16 + 32) 2^-22 of what is added, one term of du (2^-11 for
    bfloat16, else 2^-20) and of the groups' weights, one rounding."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(5)
    m, n, t = 70, 136, 4
    codes, E, scale, off = make_layer(name, m, n, group, 5)
    scale, off = scale * np.float32(200), off * np.float32(200)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=group or None)
    dy = torch.from_numpy(g.standard_normal((t, m)).astype(np.float32)).cuda()
    dy[0] *= 1e-35
    dy[0, ::2] = 0.0
    dy[1] *= 1e-36
    dy[2] = 0.0
    dy = dy.to(dtype_of(dtype))
    x = torch.from_numpy(g.standard_normal((t, n)).astype(np.float32)).cuda().to(dtype_of(dtype))
    r = mpq.linear_backward(dy, x, layer)
    want = R.linear_backward(f64(dy), f64(x), codes, E, scale, off, group)
    e, col = R.layer_entries(codes, E, group)
    mid = float(E[len(E) // 2, 0]) if E.shape[1] == 1 else 0.0
    a, o = (np.asarray(v, np.float64).reshape(m, -1)[:, col] for v in (scale, off))
    parts = np.abs(a * (e - mid)) + np.abs(o + a * mid)
    one = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
    lim = ((m / 16 + 32) * 2.0 ** -22 + 2 * one) * (np.abs(f64(dy)) @ parts)
    err = np.abs(f64(r["dx"]) - want["dx"])
    assert (err <= lim + STEP[dtype] * (np.abs(want["dx"]) + lim) + 1e-40).all(), err.max()
