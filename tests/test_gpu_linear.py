"""A packed layer's product and its gradients against float64, over codebooks,
types, groups, sizes and strides.

Tolerances, per output, with S = sum |x_j a e_j| + |o'| sum |x_j| + |bias| the
sum of the magnitudes that were added (o' the offset with the middle level):
  - float32 sums: each of the n / 16 + 32 additions that follow each other
    (matrix instructions of 32 products, their joining, the affine) may round by
    2^-24 of the partial sum, twice that inside an instruction:
    (n / 16 + 32) 2^-22 S;
  - one rounding of the result, STEP |y|;
  - what enters as float16 terms: one term rounds by 2^-11 (weights of column
    groups against bfloat16 x, many tokens), two by 2^-22 (those weights against
    the other types, float32 x; the product of two second terms that is left
    out is as small): 2^-20 in all; elements below 2^-28 of their row's largest
    lose up to 2^-39 of it, less than one addition's rounding;
  - an activation multiplies the error of its argument by its slope (below
    1.2) and adds 2^-20 (|u| + 1), its own error.
Gradients: du carries 2^-20 |dy| from the slope; dx rounds du (times scale) to one
float16 term (bfloat16: 2^-11) or two (2^-22, 2^-20 with the weights'); the sums
of the layer's gradients run over t tokens and a group's columns, du and x in two
terms at most: 2^-20.
"""
import numpy as np
import pytest

import mpq_synth as S
from oracle import ops_oracle as R
from parity_helpers import dev, host

pytestmark = pytest.mark.gpu

STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TERMS = {"bf16": 2.0 ** -11, "fp16": 2.0 ** -20, "fp32": 2.0 ** -20}


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def book(name):
    if name.startswith("s"):
        return np.arange(int(name[1:]), dtype=np.float32)[:, None]
    if name == "levels":        # a grid that is not 0 .. K - 1, exact about its middle
        return np.array([[-2.0], [-0.75], [0.0], [0.5], [3.0]], np.float32)
    if name == "vec":           # some points of E8 in another order
        return np.ascontiguousarray(S.e8_codebook(700)[::-1][:300])
    return S.e8_codebook(int(name[2:]))


def make_layer(name, m, n, group, seed, offset=True):
    g = np.random.default_rng(seed)
    E = book(name)
    d = E.shape[1]
    codes = g.integers(0, len(E), (m, n // d)).astype(np.int32)
    G = -(-n // group) if 0 < group < n else 1
    shape = (m, G) if 0 < group < n else (m,)
    scale = (0.5 + g.random(shape)).astype(np.float32) / np.sqrt(n).astype(np.float32)
    off = (scale * (g.standard_normal(shape) - (len(E) / 2 if d == 1 else 0))).astype(np.float32) if offset else None
    return codes, E, scale, off


def rows(g, t, n, dtype, pad=0, shift=0, scale=1.0):
    import torch
    buf = torch.from_numpy((g.standard_normal(t * (n + pad) + shift + 8) * scale).astype(np.float32)).cuda()
    return torch.as_strided(buf.to(dtype_of(dtype)), (t, n), (n + pad, 1), shift)


def magnitudes(x, codes, E, scale, off, group, bias=None):
    """S of the tolerances, t x m, and sum |x w|."""
    e, col = R.layer_entries(codes, E, group)
    mid = float(E[len(E) // 2, 0]) if E.shape[1] == 1 else 0.0
    a = np.asarray(scale, np.float64).reshape(len(codes), -1)[:, col]
    o = (np.asarray(off, np.float64).reshape(len(codes), -1)[:, col] if off is not None else 0.0) + a * mid
    ax = np.abs(x)
    S_ = ax @ (np.abs(a * (e - mid)) + np.abs(o)).T
    if bias is not None:
        S_ = S_ + np.abs(bias)
    return S_, ax @ np.abs(R.layer_weights(codes, E, scale, off, group)).T


def f64(t):
    return t.detach().double().cpu().numpy()


def run_case(name, m, n, t, dtype, group=0, act=None, bias=False, residual=False, offset=True, pad=0, shift=0, seed=0,
             workspace=None):
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(1000 + seed)
    codes, E, scale, off = make_layer(name, m, n, group, seed, offset)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off) if off is not None else None, group=group or None)
    x = rows(g, t, n, dtype, pad, shift)
    b = g.standard_normal(m).astype(np.float32) if bias else None
    res = rows(g, t, m, dtype, pad, shift) if residual else None
    out = rows(g, t, m, dtype, pad, shift)
    y, pre = mpq.linear(x, layer, bias=dev(b) if bias else None, activation=act, residual=res, return_pre=True, out=out,
                        workspace=workspace)
    torch.cuda.synchronize()
    assert y is out
    xr = f64(x)
    w = R.layer_weights(codes, E, scale, off, group)
    want, u = R.linear(xr, w, b, act, f64(res) if residual else None)
    S_, XW = magnitudes(xr, codes, E, scale, off, group, b)
    tol = ((n / 16 + 32) * 2.0 ** -22 + (2.0 ** -20 if dtype == "fp32" else 0.0)) * S_
    if 0 < group < n:
        tol = tol + TERMS[dtype] * XW
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    err = np.abs(f64(pre) - u)
    assert (err <= tol + STEP[dtype] * np.abs(u) + tiny).all(), ("pre", (err / (tol + STEP[dtype] * np.abs(u))).max())
    tol_y = 1.2 * tol + (2.0 ** -20 * (np.abs(u) + 1) if act else 0)
    lim = tol_y + STEP[dtype] * (np.abs(want) + tol_y) + 2.0 ** -24 * np.abs(u) + tiny
    err = np.abs(f64(y) - want)
    assert (err <= lim).all(), ("y", (err / lim).max())
    return layer, x, pre


BOOKS = ["s2", "s3", "s8", "s16", "s17", "s64", "levels", "vec", "e865536", "e81", "e8240", "e8241", "e81000", "e82401",
         "e830000", "e856881"]


@pytest.mark.parametrize("name", BOOKS)
@pytest.mark.parametrize("t", [3, 130])
def test_linear_books(name, t):
    run_case(name, 70, 136, t, "bf16", act="silu", bias=True, residual=True, seed=len(name) + t)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,m,n", [("s16", 1, 1), ("s8", 17, 65), ("s64", 33, 127), ("e865536", 16, 8),
                                      ("e865536", 300, 1032), ("s16", 520, 700)])
@pytest.mark.parametrize("t", [1, 2, 17, 33, 65, 129, 300])
def test_linear_sizes(dtype, name, m, n, t):
    run_case(name, m, n, t, dtype, bias=True, seed=m + n + t)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,n,group", [("s16", 512, 128), ("s16", 500, 128), ("s64", 320, 64), ("s16", 200, 33),
                                          ("s8", 96, 1), ("s16", 256, 256), ("s16", 100, 4096)])
@pytest.mark.parametrize("t", [1, 20, 140])
def test_linear_groups(dtype, name, n, group, t):
    run_case(name, 50, n, t, dtype, group=group, act="gelu_tanh", seed=n + group + t)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,m,n,group", [
    ("s16", 1, 1, 0), ("s8", 17, 65, 0), ("s64", 33, 127, 0), ("e865536", 16, 8, 0), ("e830000", 70, 136, 0),
    ("vec", 70, 136, 0), ("levels", 130, 200, 0), ("s16", 50, 512, 128), ("s16", 50, 500, 128), ("s64", 50, 320, 64)])
def test_linear_many_tokens(dtype, name, m, n, group):
    """More tokens than the packed codes are ever read for."""
    run_case(name, m, n, 1030, dtype, group=group, act="silu", bias=True, residual=True, seed=m + n)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8)])
def test_linear_many_tokens_strides(dtype, pad, shift):
    run_case("e865536", 131, 128, 1025, dtype, residual=True, pad=pad, shift=shift)
    run_case("s16", 64, 129, 1025, dtype, residual=True, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype,t,group", [("bf16", 128, 0), ("bf16", 129, 0), ("bf16", 192, 0),
                                           ("bf16", 193, 0), ("fp32", 96, 0), ("fp32", 97, 0),
                                           ("bf16", 192, 128), ("bf16", 193, 128), ("fp16", 384, 128),
                                           ("fp16", 385, 128)])
def test_linear_either_side_of_the_packed_codes(dtype, t, group):
    """A layer large enough that the token count decides, at the counts where it does."""
    run_case("s16", 2050, 2176, t, dtype, group=group, bias=True)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_linear_activations(act):
    run_case("s16", 64, 256, 9, "fp32", act=act, bias=True, residual=True)
    run_case("s16", 64, 256, 200, "fp32", act=act, bias=True, residual=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (5, 4)])
@pytest.mark.parametrize("t", [5, 150])
def test_linear_strides(dtype, pad, shift, t):
    run_case("e865536", 131, 128, t, dtype, residual=True, pad=pad, shift=shift)
    run_case("s16", 64, 129, t, dtype, residual=True, pad=pad, shift=shift)


@pytest.mark.parametrize("t", [1, 64, 200])
def test_linear_no_offset_and_many_tiles(t):
    run_case("e865536", 9000, 64, t, "bf16", offset=False)
    run_case("s16", 9000, 64, t, "bf16", offset=False)


def test_linear_large():
    """The product of a large layer, one column of the output per check: sums of 14336."""
    run_case("e865536", 272, 14336, 2, "bf16", residual=True, offset=False)
    run_case("e865536", 272, 14336, 270, "bf16", residual=True, offset=False)


def test_linear_in_place_residual_and_rows_left_alone():
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 48, 160, 0, 3)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    for t in (4, 140):
        x = torch.randn(t, 160, device="cuda").bfloat16()
        buf = torch.randn(t + 3, 50, device="cuda").bfloat16()
        before = buf.clone()
        want = mpq.linear(x, layer, residual=before[:t, :48])
        got = mpq.linear(x, layer, residual=buf[:t, :48], out=buf[:t, :48])
        assert got.data_ptr() == buf.data_ptr() and torch.equal(buf[:t, :48], want)
        assert torch.equal(buf[t:], before[t:]) and torch.equal(buf[:, 48:], before[:, 48:])


def test_linear_nonfinite_among_many_tokens():
    import torch
    import post_quantization_solver_amd as mpq
    for name, group in (("e865536", 0), ("s16", 128)):
        codes, E, scale, off = make_layer(name, 48, 256, group, 4)
        layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=group or None)
        for dtype in ("bf16", "fp16", "fp32"):
            x = torch.randn(1030, 256, device="cuda").to(dtype_of(dtype))
            clean = mpq.linear(x, layer)
            x[3, 7], x[1029, 100] = float("nan"), float("inf")
            y = mpq.linear(x, layer)
            keep = [i for i in range(1030) if i not in (3, 1029)]
            assert torch.equal(y[keep], clean[keep])
            assert torch.isnan(y[3]).all() and not torch.isfinite(y[1029]).any()


def test_linear_nonfinite_tokens_stay_apart():
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("e865536", 48, 160, 0, 4)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    for dtype in ("bf16", "fp32"):
        for t in (18, 140):
            x = torch.randn(t, 160, device="cuda").to(dtype_of(dtype))
            clean = mpq.linear(x, layer)
            x[3, 7], x[17, 100] = float("nan"), float("inf")
            y = mpq.linear(x, layer)
            keep = [i for i in range(t) if i not in (3, 17)]
            assert torch.equal(y[keep], clean[keep])
            assert torch.isnan(y[3]).all() and not torch.isfinite(y[17]).any()


def run_grad(name, m, n, t, dtype, group=0, act=None, offset=True, pad=0, shift=0, seed=0):
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(2000 + seed)
    codes, E, scale, off = make_layer(name, m, n, group, seed, offset)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off) if off is not None else None, group=group or None)
    x = rows(g, t, n, dtype, pad, shift)
    dy = rows(g, t, m, dtype, pad, shift, 0.1)
    pre = rows(g, t, m, dtype, pad, shift, 1.5) if act else None
    r = mpq.linear_backward(dy, x, layer, pre=pre, activation=act)
    torch.cuda.synchronize()
    xr, dyr, prer = f64(x), f64(dy), f64(pre) if act else None
    want = R.linear_backward(dyr, xr, codes, E, scale, off, group, prer, act)
    w = np.abs(R.layer_weights(codes, E, scale, off, group))
    e, col = R.layer_entries(codes, E, group)
    mid = float(E[len(E) // 2, 0]) if E.shape[1] == 1 else 0.0
    a = np.asarray(scale, np.float64).reshape(m, -1)[:, col]
    o = (np.asarray(off, np.float64).reshape(m, -1)[:, col] if off is not None else 0.0) + a * mid
    du = np.abs(dyr * (R.act_slope(act, prer) if act else 1.0))
    slope = 2.0 ** -20 * np.abs(dyr) if act else 0.0
    parts = np.abs(a * (e - mid)) + np.abs(o)
    one = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20
    lim = ((m / 16 + 32) * 2.0 ** -22 + one) * (du @ parts) + (slope * np.ones_like(du)) @ parts
    if 0 < group < n:
        lim = lim + TERMS[dtype] * (du @ w)
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    err, top = np.abs(f64(r["dx"]) - want["dx"]), lim + STEP[dtype] * (np.abs(want["dx"]) + lim) + tiny
    assert (err <= top).all(), ("dx", (err / top).max())
    G = int(col[-1]) + 1
    dW = ((t / 16 + 32) * 2.0 ** -22 + 2.0 ** -20) * (du.T @ np.abs(xr)) + ((slope * np.ones_like(du)).T @ np.abs(xr))
    for key, fac in (("dscale", np.abs(e)), ("doffset", np.ones_like(e))):
        top = np.zeros((m, G))
        for k in range(G):
            top[:, k] = (dW * fac)[:, col == k].sum(1)
        top = top.reshape(np.shape(scale)) + 2.0 ** -23 * np.abs(want[key])
        err = np.abs(f64(r[key]) - want[key])
        assert r[key].shape == scale.shape and (err <= top).all(), (key, (err / top).max())
    err = np.abs(f64(r["dbias"]) - want["dbias"])
    assert (err <= 2.0 ** -17 * du.sum(0) + (slope * np.ones_like(du)).sum(0) + 1e-30).all()
    # halves of the call
    a1 = mpq.linear_backward(dy, x, layer, pre=pre, activation=act, need_dlayer=False)
    a2 = mpq.linear_backward(dy, x, layer, pre=pre, activation=act, need_dx=False)
    assert a1["dscale"] is None and a2["dx"] is None
    assert torch.equal(a1["dx"], r["dx"]) and all(torch.equal(a2[k], r[k]) for k in ("dscale", "doffset", "dbias"))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,m,n,t,group,act", [
    ("s16", 1, 1, 1, 0, None), ("s16", 70, 130, 3, 0, "gelu"), ("s64", 33, 127, 65, 0, "silu"),
    ("e865536", 65, 136, 64, 0, None), ("e81000", 200, 72, 100, 0, "gelu_tanh"), ("vec", 64, 64, 17, 0, "relu"),
    ("s16", 70, 260, 40, 128, None), ("s16", 31, 100, 40, 7, "silu"), ("s8", 16, 64, 200, 64, "gelu"),
    ("levels", 129, 257, 5, 0, None)])
def test_linear_backward(dtype, name, m, n, t, group, act):
    run_grad(name, m, n, t, dtype, group, act, seed=m + n)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_backward_strides_and_no_offset(dtype):
    run_grad("e865536", 50, 64, 20, dtype, pad=3, shift=1, offset=False, act="silu")
    run_grad("s16", 300, 640, 700, dtype, offset=False)


def test_linear_backward_differences():
    """Against central differences of the forward pass in float32."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(9)
    codes, E, scale, off = make_layer("s16", 12, 40, 16, 9)
    x = rows(g, 6, 40, "fp32").clone()
    b = g.standard_normal(12).astype(np.float32)
    v = rows(g, 6, 12, "fp32")

    def loss(x_, s_, o_, b_):
        layer = mpq.pack_layer(dev(codes), E, s_, o_, group=16)
        return float((mpq.linear(x_, layer, bias=b_, activation="gelu").double() * v.double()).sum())
    args = [x, dev(scale), dev(off), dev(b)]
    layer = mpq.pack_layer(dev(codes), E, args[1], args[2], group=16)
    _, pre = mpq.linear(x, layer, bias=args[3], activation="gelu", return_pre=True)
    r = mpq.linear_backward(v, x, layer, pre=pre, activation="gelu")
    for k, key in enumerate(("dx", "dscale", "doffset", "dbias")):
        flat = r[key].flatten()
        for at in (0, flat.numel() // 2, flat.numel() - 1):
            h = 2.0 ** -7 if key in ("dx", "dbias") else 2.0 ** -10
            up, dn = [a.clone() for a in args], [a.clone() for a in args]
            up[k].view(-1)[at] += h
            dn[k].view(-1)[at] -= h
            d = (loss(*up) - loss(*dn)) / (2 * h)
            # the third derivative of the loss along one parameter: the gelu's (below 2) times the cube of the
            # argument's slope (at most 16 x 8 x 4 for scale and offset), over six tokens
            ref = float(flat[at])
            assert abs(d - ref) <= 2e-2 * max(1.0, abs(ref)), (key, at, d, ref)


def test_linear_empty():
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 20, 33, 0, 1)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    x = torch.empty(0, 33, device="cuda")
    assert mpq.linear(x, layer).shape == (0, 20)
    r = mpq.linear_backward(torch.empty(0, 20, device="cuda"), x, layer)
    assert r["dx"].shape == (0, 33) and all(float(r[k].abs().max()) == 0 for k in ("dscale", "doffset", "dbias"))
    none = mpq.pack_layer(dev(codes[:0]), E, dev(scale[:0]), dev(off[:0]))
    assert mpq.linear(torch.randn(3, 33, device="cuda"), none).shape == (3, 0)


def test_linear_is_deterministic_and_follows_the_affine():
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("e865536", 256, 512, 0, 5)
    s = dev(scale)
    layer = mpq.pack_layer(dev(codes), E, s)
    x = torch.randn(7, 512, device="cuda").bfloat16()
    y = mpq.linear(x, layer)
    assert torch.equal(y, mpq.linear(x, layer))
    s.mul_(2)    # the layer holds the tensor itself
    assert torch.equal(mpq.linear(x, layer).float(), y.float() * 2)


@pytest.mark.parametrize("t", [5, 140])
def test_linear_graph_replays(t):
    """Two captured graphs of calls in turn, replayed on new inputs with eager work between."""
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 200, 384, 128, 6)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=128)
    x = torch.randn(t, 384, device="cuda").bfloat16()
    dy = torch.randn(t, 200, device="cuda").bfloat16()

    def fwd():
        return list(mpq.linear(x, layer, activation="silu", return_pre=True))

    def bwd():
        r = mpq.linear_backward(dy, x, layer, pre=mpq.linear(x, layer, activation="silu", return_pre=True)[1],
                                activation="silu")
        return [r[k] for k in ("dx", "dscale", "doffset", "dbias")]
    fwd(), bwd()
    torch.cuda.synchronize()
    graphs = []
    for fn in (fwd, bwd):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = fn()
        graphs.append((gr, out, fn))
    for k in range(3):
        x.copy_(torch.randn(t, 384, device="cuda"))
        dy.copy_(torch.randn(t, 200, device="cuda"))
        torch.cuda.synchronize()
        for gr, out, fn in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, fn()):
                assert torch.equal(a, b), k


@pytest.mark.parametrize("name,t", [("e865536", 1), ("e865536", 40), ("e865536", 1030), ("s16", 1), ("s16", 1030)])
def test_linear_graph_replays_on_every_path(name, t):
    """A chain of calls captured, replayed on new inputs and a tuned scale, with eager work between."""
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer(name, 256, 256, 0, 6)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    x = torch.randn(t, 256, device="cuda").bfloat16()

    def chain():
        h = mpq.linear(x, layer, activation="silu")
        y = mpq.linear(h, layer, residual=x)
        r = mpq.linear_backward(y, x, layer)
        return [h, y, r["dx"], r["dscale"], r["doffset"], r["dbias"]]
    chain()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = chain()
    for k in range(3):
        x.copy_(torch.randn(t, 256, device="cuda"))
        layer.scale.mul_(1.25)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, chain()):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("t", [1, 20, 1100])
def test_linear_two_streams_at_once(t):
    """Calls on two streams that overlap: each has its own workspace, and the results are the serial ones."""
    import torch
    import post_quantization_solver_amd as mpq
    layers = []
    for seed, name in ((1, "e865536"), (2, "s16")):
        codes, E, scale, off = make_layer(name, 1024, 1024, 0, seed)
        layers.append(mpq.pack_layer(dev(codes), E, dev(scale), dev(off)))
    xs = [torch.randn(t, 1024, device="cuda").bfloat16() for _ in layers]
    want = [mpq.linear(x, layer, activation="gelu") for x, layer in zip(xs, layers)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(mpq.linear(xs[k], layers[k], activation="gelu"))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(g, want[k]) for g in got[k])


@pytest.mark.parametrize("name,half", [("e865536", 0.5), ("s16", 1.0), ("s64", 1.0)])
@pytest.mark.parametrize("t", [1, 17, 70])
def test_linear_outliers_in_x(name, half, t):
    """One element of a token 2^14 times the others.  Lifted entries: a unit's sum of up to 191 (E8: 143 half units)
    |x| and its lift come off each other, some six roundings of 2^-24 of 351 (E8: 140) |x| at most: 2^-13 a sum |x|."""
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, _ = make_layer(name, 96, 1024, 0, 7, False)
    layer = mpq.pack_layer(dev(codes), E, dev(scale))
    x = torch.randn(t, 1024, device="cuda").bfloat16()
    x[:, 300] = 16384.0
    got = f64(mpq.linear(x, layer))
    xr = f64(x)
    want = xr @ R.layer_weights(codes, E, scale, None, 0).T
    step = half * 2 if name.startswith("e8") else float(E[1, 0] - E[0, 0])
    tol = 2.0 ** -13 * np.abs(xr).sum(1)[:, None] * np.abs(scale)[None, :] * step
    assert (np.abs(got - want) <= tol + STEP["bf16"] * (np.abs(want) + tol)).all()


def test_solve_run_score_tune():
    """The operators together: a solved layer as an output head, its logits scored and tuned to the original's."""
    import torch
    import post_quantization_solver_amd as mpq
    L = S.make_layer("head", 512, 128, seed=91, d=1, bits=3, power=0.5, T_vamp=4)
    T = {k: dev(getattr(L, k)) for k in ("W", "s", "V", "a", "o")}
    cb = mpq.prepare_codebook(L.E)
    codes = mpq.quantize_layer(T["W"], T["s"], T["V"], cb, T["a"], T["o"], T_vamp=4, n_cd=2)["codes"]
    layer = mpq.pack_layer(codes, cb, T["a"], T["o"])
    x = (torch.randn(48, 128, device="cuda") * 0.2)
    teacher = (x.double() @ T["W"].double().T).float()
    top = mpq.token_logprobs(teacher, top=64)
    weights = torch.full((48,), 1 / 48, device="cuda")
    logits = mpq.linear(x, layer)
    first = mpq.token_logprobs(logits, top["top_ids"][:, 0].contiguous())
    r = mpq.distill(logits, top["top_ids"], top["top_logprobs"], tail=True, weights=weights)
    grads = mpq.linear_backward(r["grad"], x, layer)
    # against float64 autograd over the layer's scale and offset
    E = torch.from_numpy(L.E).double()
    a, o = (v.double().cpu().requires_grad_() for v in (T["a"], T["o"]))
    W = a[:, None] * E[codes.cpu().long()].reshape(512, 128) + o[:, None]
    z = x.double().cpu() @ W.T
    lq = torch.log_softmax(z, 1)
    lp, ids = top["top_logprobs"].double().cpu(), top["top_ids"].long().cpu()
    rest = 1 - lp.exp().sum(1)
    hidden = torch.zeros_like(lq, dtype=torch.bool).scatter_(1, ids, True)
    lq_rest = torch.logsumexp(lq.masked_fill(hidden, -np.inf), 1)
    kl = (lp.exp() * (lp - lq.gather(1, ids))).sum(1) + rest * (rest.log() - lq_rest)
    (kl / 48).sum().backward()
    assert float((r["loss"].double().cpu() - kl.detach() / 48).abs().max()) < 1e-6
    assert float((first["logprob"].double().cpu() - lq.detach().gather(1, ids[:, :1])[:, 0]).abs().max()) < 1e-4
    for got, ref in ((grads["dscale"], a.grad), (grads["doffset"], o.grad)):
        assert float((got.double().cpu() - ref).norm() / ref.norm()) < 1e-4


def test_linear_refusals():
    import torch
    import post_quantization_solver_amd as mpq
    codes, E, scale, off = make_layer("s16", 20, 32, 0, 1)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    x = torch.randn(3, 32, device="cuda")
    with pytest.raises(TypeError):
        mpq.linear(x.double(), layer)
    with pytest.raises(ValueError):
        mpq.linear(x[:, :31], layer)
    with pytest.raises(ValueError):
        mpq.linear(torch.randn(32, 3, device="cuda").t(), layer)
    with pytest.raises(ValueError):
        mpq.linear(x, layer, activation="tanh")
    with pytest.raises(ValueError):
        mpq.linear(x, layer, bias=torch.zeros(19, device="cuda"))
    with pytest.raises(TypeError):
        mpq.linear(x, layer, bias=torch.zeros(20, device="cuda").half())
    with pytest.raises(TypeError):
        mpq.linear(x, layer, residual=torch.zeros(3, 20, device="cuda").half())
    with pytest.raises(TypeError):
        mpq.linear(x.cpu(), layer)
    with pytest.raises(ValueError):
        mpq.linear_backward(torch.zeros(3, 20, device="cuda"), x, layer, activation="silu")
    with pytest.raises(mpq.MPQError):
        mpq.linear(x, layer, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mpq.MPQError):      # levels that 16 bits do not hold
        mpq.pack_layer(dev(codes), np.linspace(0, 1, 16, dtype=np.float32)[:, None] ** 2, dev(scale), dev(off))
    with pytest.raises(mpq.MPQError):
        c8, E8, s8, _ = make_layer("e81000", 4, 32, 0, 1)
        mpq.pack_layer(dev(c8), E8, dev(s8), group=16)
    with pytest.raises(ValueError):
        mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=16)
    with pytest.raises(TypeError):
        mpq.pack_layer(dev(codes).long(), E, dev(scale), dev(off))


def test_backward_of_the_longest_layer():
    """2^24 rows: a tile's planes span more than 4 GB.  du is not zero in ten rows alone, so the sums are theirs."""
    import torch
    import post_quantization_solver_amd as mpq
    m, n = 1 << 24, 144
    E = (np.arange(16, dtype=np.float32) - 8).reshape(16, 1)
    codes = torch.randint(0, 16, (m, n), dtype=torch.int32, device="cuda")
    scale = torch.ones(m, device="cuda")
    layer = mpq.pack_layer(codes, E, scale)
    at = torch.linspace(0, m - 1, 10, device="cuda").long()
    dy = torch.zeros((1, m), dtype=torch.bfloat16, device="cuda")
    dy[0, at] = torch.arange(1, 11, device="cuda").bfloat16()
    entries = codes[at].double().cpu().numpy() - 8
    del codes
    x = torch.zeros((1, n), dtype=torch.bfloat16, device="cuda")
    dx = f64(mpq.linear_backward(dy, x, layer, need_dlayer=False)["dx"])
    want = np.arange(1, 11) @ entries   # integers below 2^24: exact but for dx's own rounding
    assert (np.abs(dx[0] - want) <= STEP["bf16"] * np.abs(want)).all()
