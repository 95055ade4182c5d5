"""The products' large tiles (taken from 192 of them on), their ragged edges, fewer
steps than stages and the steady state, and layers that go through the workspace in
blocks of rows: parity against float64 with the tolerances of test_gpu_linear.py."""
import numpy as np
import pytest

from oracle import ops_oracle as R
from parity_helpers import dev
from test_gpu_linear import STEP, f64, make_layer, rows, run_case, run_grad

pytestmark = pytest.mark.gpu


# 256 x 128 at 2050 x 3100 (9 x 25 tiles), 256 x 256 at 4100 x 3400 (17 x 14); three steps a plane pair or four, fewer
# than stages, and the steady state with an odd and an even count of steps
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,t", [(2050, 3100), (4100, 3400)])
@pytest.mark.parametrize("name,n,group", [("e865536", 96, 0), ("s16", 64, 0), ("s16", 129, 0), ("s16", 120, 33),
                                          ("s64", 544, 64)])
def test_forward_tiles(dtype, m, t, name, n, group):
    run_case(name, m, n, t, dtype, group=group, act="silu", bias=True, residual=True, seed=n)


@pytest.mark.parametrize("m,t", [(2050, 3100), (4100, 3400)])
def test_forward_tiles_steady_state(m, t):
    run_case("e865536", m, 1056, t, "bf16", residual=True, pad=3, shift=1)


# dx: 2060 columns x 3080 tokens (9 x 25), 4100 x 3400 (17 x 14)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,t", [(2056, 3080), (4104, 3400)])
@pytest.mark.parametrize("name,m,group,act", [("e865536", 96, 0, None), ("s16", 65, 128, "silu")])
def test_dx_tiles(dtype, n, t, name, m, group, act):
    run_grad(name, m, n, t, dtype, group, act, seed=n + m)


# the layer's gradients: n x m as above, contracted (rows, groups of 64 columns' multiples) or formed (33 columns)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,m", [(2056, 3080), (4104, 3400)])
@pytest.mark.parametrize("name,t,group,act", [("e865536", 40, 0, None), ("s16", 300, 0, "gelu"), ("s16", 70, 512, None),
                                              ("s64", 130, 700, None)])
def test_contraction_tiles(dtype, n, m, name, t, group, act):
    run_grad(name, m, n, t, dtype, group, act, seed=n + t)


def test_forward_blocks_of_rows():
    """Layers whose planes take more than 128 MB: entries (1024 rows a block), and weights in two terms (2304)."""
    run_case("e865536", 1100, 65536, 130, "bf16", bias=True, residual=True, act="relu")
    run_case("s16", 2500, 14336, 5, "fp16", group=100, bias=True, residual=True, act="relu")


def test_gradients_blocks_of_rows():
    """dW of groups of 33 columns, formed 512 rows at a time."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(77)
    m, n, t, group = 600, 65536, 5, 33
    codes, E, scale, off = make_layer("s16", m, n, group, 3)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=group)
    x, dy, pre = rows(g, t, n, "fp16"), rows(g, t, m, "fp16", scale=0.1), rows(g, t, m, "fp16", scale=1.5)
    r = mpq.linear_backward(dy, x, layer, pre=pre, activation="silu")
    torch.cuda.synchronize()
    xr, dyr = f64(x), f64(dy)
    du = dyr * R.act_slope("silu", f64(pre))
    dW, e = du.T @ xr, E[:, 0].astype(np.float64)[codes]
    top = (((t / 16 + 32) * 2.0 ** -22 + 2.0 ** -20) * np.abs(du).T + 2.0 ** -20 * np.abs(dyr).T) @ np.abs(xr)
    starts = np.arange(0, n, group)
    for key, fac in (("dscale", e), ("doffset", 1.0)):
        want = np.add.reduceat(dW * fac, starts, axis=1)
        lim = np.add.reduceat(top * fac, starts, axis=1) + 2.0 ** -23 * np.abs(want)
        err = np.abs(f64(r[key]) - want)
        assert r[key].shape == want.shape and (err <= lim).all(), (key, (err / lim).max())
    assert (np.abs(f64(r["dbias"]) - du.sum(0)) <= 2.0 ** -17 * np.abs(du).sum(0) + 2.0 ** -20 * np.abs(dyr).sum(0)).all()
    w = np.repeat(scale.astype(np.float64), group, 1)[:, :n] * e + np.repeat(off.astype(np.float64), group, 1)[:, :n]
    want, mag = du @ w, np.abs(du) @ np.abs(w)
    # the sums' magnitudes: entries about the middle level and the offset there, each at most their own weight's
    mid = float(E[8, 0])
    a, o = (np.repeat(v.astype(np.float64), group, 1)[:, :n] for v in (scale, off))
    parts = np.abs(a * (e - mid)) + np.abs(o + a * mid)
    lim = ((m / 16 + 32) * 2.0 ** -22 + 2.0 ** -20) * (np.abs(du) @ parts) + 2.0 ** -20 * (np.abs(dyr) @ parts + mag)
    err = np.abs(f64(r["dx"]) - want)
    assert (err <= lim + STEP["fp16"] * (np.abs(want) + lim) + 2.0 ** -25).all(), (err / lim).max()


# 4100 rows are 257 tiles of sixteen: five tiles of tokens a workgroup take two rounds of the card where four take three
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("name,n,group", [("e865536", 264, 0), ("e8241", 40, 0), ("s16", 130, 0), ("s64", 257, 0),
                                          ("levels", 200, 0), ("vec", 136, 0), ("s16", 500, 128), ("s64", 320, 64),
                                          ("levels", 256, 128)])
@pytest.mark.parametrize("t", [65, 80, 145])
def test_five_tiles_of_tokens(dtype, name, n, group, t):
    run_case(name, 4100, n, t, dtype, group=group, act="silu", bias=True, residual=True, seed=n + t)
