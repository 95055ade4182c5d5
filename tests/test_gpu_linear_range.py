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


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_slopes_far_out(act, dtype):
    """Arguments beyond float16 are kept as infinities: their slopes are 0 and 1, as the activation's finite values
    there say, and a NaN stays one.  d bias of one token is du itself: the slope, exact at both ends (2^-20 where it
    is not: the activation's own error)."""
    import torch
    import post_quantization_solver_amd as mpq
    far = 65504.0 if dtype == "fp16" else 3e38
    pre = torch.tensor([[-np.inf, np.inf, -far, far, -300.0, 300.0, -40.0, 40.0, 0.0, np.nan]], device="cuda")
    m = pre.shape[1]
    codes, E, scale, off = make_layer("s16", m, 32, 0, 1)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    one = torch.ones(1, m, device="cuda").to(dtype_of(dtype))
    x = torch.ones(1, 32, device="cuda").to(dtype_of(dtype))
    r = mpq.linear_backward(one, x, layer, pre=pre.to(dtype_of(dtype)), activation=act)
    got = f64(r["dbias"])
    assert np.isnan(got[-1]) and np.isfinite(got[:-1]).all(), got
    assert np.array_equal(got[:6], [0, 1, 0, 1, 0, 1])
    half = 0.0 if act == "relu" else 0.5
    assert np.abs(got[6:9] - [0, 1, half]).max() <= 2.0 ** -20
    y = f64(mpq.linear_backward(one[:, :-1].contiguous(), x, mpq.pack_layer(dev(codes[:-1]), E, dev(scale[:-1]),
            dev(off[:-1])), pre=pre[:, :-1].contiguous().to(dtype_of(dtype)), activation=act)["dx"])
    assert np.isfinite(y).all()


def test_levels_that_both_16_bit_types_hold():
    """pack_layer takes differences to the middle level that bfloat16 and float16 hold, subnormal ones too, and no
    others."""
    import torch
    import post_quantization_solver_amd as mpq
    codes = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    scale = torch.ones(2, device="cuda")
    for low, taken in ((2.0 ** -24, True), (2.0 ** -25, False), (1.5 * 2.0 ** -24, False), (3 * 2.0 ** -24, True),
                       (2.0 ** -14, True), (65280.0, True), (65536.0, False), (1 + 2.0 ** -7, True),
                       (1 + 2.0 ** -8, False), (float(np.float32(0.1)), False)):
        for x in (low, -low):
            E = np.array([[x], [0.0]] if x < 0 else [[0.0], [0.0], [x]], np.float32)
            if taken:
                mpq.pack_layer(codes, E, scale)
            else:
                with pytest.raises(mpq.MPQError):
                    mpq.pack_layer(codes, E, scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_of_a_layer_without_rows(dtype):
    """dx is zeros, in its own elements alone; nothing else has an element."""
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 4, 33, 0, 1)
    none = mpq.pack_layer(dev(codes[:0]), E, dev(scale[:0]), dev(off[:0]))
    x = torch.ones(70, 33, device="cuda").to(dtype_of(dtype))
    r = mpq.linear_backward(x[:, :0], x, none)
    assert r["dx"].shape == (70, 33) and not r["dx"].any() and r["dscale"].shape == (0,) == r["dbias"].shape
    buf = torch.ones(70, 40, device="cuda").to(dtype_of(dtype))
    lib = mpq.load_library()
    code = {"bf16": 0, "fp32": 2}[dtype]
    assert lib.mpq_linear_backward(None, 0, x.data_ptr(), code, 70, 33, None, 0, 33, none.codebook.ref(), None, None, 0,
                                   0, None, 0, buf.data_ptr(), 40, None, None, None, None, 0,
                                   torch.cuda.current_stream().cuda_stream) == 0
    assert not buf[:, :33].any() and (buf[:, 33:] == 1).all()


@pytest.mark.parametrize("group", [0, 16])
def test_a_replaced_affine_is_checked(group):
    """scale and offset of a packed layer are public: others of their kind are used, anything else is refused."""
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 20, 64, group, 1)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=group or None)
    x, dy = torch.randn(3, 64, device="cuda"), torch.randn(3, 20, device="cuda")
    y = mpq.linear(x, layer)
    good = {"scale": dev(scale), "offset": dev(off)}
    for name, t in good.items():
        for bad in (t.half(), t.double(), t.cpu(), None if name == "scale" else 0.5, t[:19].contiguous(),
                    t.view(-1)[:1], torch.zeros(20, 3, device="cuda"), torch.zeros(40, 4, device="cuda")[::2],
                    torch.zeros(4, 20, device="cuda").t()):
            setattr(layer, name, bad)
            with pytest.raises((TypeError, ValueError)):
                mpq.linear(x, layer)
            with pytest.raises((TypeError, ValueError)):
                mpq.linear_backward(dy, x, layer)
        setattr(layer, name, t.clone())
        assert torch.equal(mpq.linear(x, layer), y)
    layer.offset = None
    assert torch.equal(mpq.linear(x, layer), mpq.linear(x, mpq.pack_layer(dev(codes), E, dev(scale), group=group or None)))
    if not group:
        layer.scale = dev(scale)[:, None]
        r = mpq.linear_backward(dy, x, layer)
        assert r["dscale"].shape == (20, 1)


def test_an_autograd_graph_does_not_end_unnoticed():
    """linear records no graph: an input that has one is refused, except where gradients are off.  The graph goes on by
    hand, through linear_backward."""
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 20, 64, 0, 1)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    leaf = torch.randn(3, 64, device="cuda", requires_grad=True)
    x, res = leaf * 2, torch.zeros(3, 20, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        mpq.linear(x, layer)
    with pytest.raises(ValueError):
        mpq.linear(leaf, layer)
    with pytest.raises(ValueError):
        mpq.linear(x.detach(), layer, residual=res)
    y = mpq.linear(x.detach(), layer, residual=res.detach())
    with torch.no_grad():
        assert torch.equal(mpq.linear(x, layer, residual=res), y)
    dx = mpq.linear_backward(y, x, layer)["dx"]
    x.backward(dx)
    assert torch.equal(leaf.grad, 2 * dx)
