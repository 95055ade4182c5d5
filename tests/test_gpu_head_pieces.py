"""Vocabularies in several pieces: which tile each piece takes, and sums over pieces of the longest rows.

The longest rows are made of numbers whose sums float32 holds exactly in any order (x of +-1, weights k 2^-8 with |k|
below 8: all sums are multiples of 2^-8 below 2^11), so that a logit is off by its last operations alone, 2^-22 of the
magnitudes of s and the bias, and not by a bound of 65536 additions, which would let anything pass.  That the tolerances
bite is shown by results that have to fail: scaled by 0.9, or without the last piece.
"""
import numpy as np
import pytest

from parity_helpers import dev
from test_gpu_head import inputs, matrix_case, packed_case, reference
from test_gpu_linear import STEP, dtype_of

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ tiles of pieces without kept logits

# 33000 tokens: pieces of 1792 rows (256 x 256 tiles), the last of 208, 256 or 8: 256 x 128 tiles.
LAST = [(1792 + 208, 33000), (1792 + 256, 32897), (1792 + 8, 33001), (2 * 1792 + 100, 33000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,t", LAST)
@pytest.mark.parametrize("need_dhead", [False, True])
def test_small_last_piece_matrix(dtype, m, t, need_dhead):
    """Rows read in place, and planes."""
    matrix_case(m, 64, t, dtype, padded=True, seed=m, need_dhead=need_dhead)
    matrix_case(m, 40, t, dtype, padded=True, seed=m, need_dhead=need_dhead)
    matrix_case(m, 128, t, dtype, pad=1, seed=m, need_dhead=need_dhead)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,t", LAST)
@pytest.mark.parametrize("name,n,group", [("s16", 40, 0), ("s64", 72, 0), ("e8240", 64, 0), ("s16", 192, 64), ("s16", 96, 32)])
def test_small_last_piece_packed(dtype, m, t, name, n, group):
    import torch
    import post_quantization_solver_amd as mpq
    head, x, targets, b, w, full = packed_case(name, m, n, t, dtype, group=group, padded=True, seed=m)
    got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dx=False, need_dhead=False)
    assert torch.equal(got["loss"], full["loss"])
    if not group:   # (dz out of the product's registers whatever is wanted)
        for need_dx, need_dhead in ((True, False), (False, True)):
            got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dx=need_dx, need_dhead=need_dhead)
            assert all(v is None or torch.equal(v, full[k]) for k, v in got.items())
    else:   # dz out of the product's registers, without the gradients of the groups
        packed_case(name, m, n, t, dtype, group=group, padded=True, seed=m, need_dhead=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_some_hundred_tokens_of_a_large_matrix(dtype, pad):
    """300 tokens of 120000 rows: every piece in tiles of 128 tokens, the last of those ragged."""
    n = 8192 if dtype == "fp32" else 16384
    m, t = (120_000 if dtype == "fp32" else 115_000), 300
    import torch
    import post_quantization_solver_amd as mpq
    from test_gpu_head import check
    gen = torch.Generator(device="cuda").manual_seed(pad)
    buf = torch.empty(m, n + pad, device="cuda", dtype=dtype_of(dtype))
    for k in range(0, m, 5000):
        buf[k:k + 5000] = torch.randn(min(5000, m - k), n + pad, generator=gen, device="cuda") * (3.0 / np.sqrt(n))
    W = buf[:, :n]
    x, targets, b, w = inputs(np.random.default_rng(pad), m, n, t, dtype, True, True, 0, 0)
    got = mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w, need_dhead=False)
    # the first and last tokens against the formula (float64 copies of the matrix are 16 GB each)
    for part in (slice(0, 20), slice(t - 20, t)):
        ref = reference(x[part], dict(W=W), targets[part], b, w[part])
        check(dict(loss=got["loss"][part], dx=got["dx"][part], dbias=None), ref, dtype, n, dtype != "fp32", "matrix",
              need_dhead=False)


# ------------------------------------------------------------------ the longest rows

N = 65536


def passes(got, ref, dtype, kind, bias, head=None):
    """Whether a result is within its tolerances: a dict of what is not (name: worst ratio)."""
    import torch
    V, t = ref["z"].shape[1], len(ref["x"])
    half, step, tiny = dtype != "fp32", STEP[dtype], 2.0 ** -25 if dtype == "fp16" else 1e-38
    s = ref["z"] - (0.0 if bias is None else bias.double())
    d = 2.0 ** -22 * (s.abs() + (0.0 if bias is None else bias.double().abs())).amax(1)
    if kind == "rows":   # a s' + o' X + b: their own roundings
        d = d + 2.0 ** -22 * head["parts"].amax(1)
    adz = ref["dz"].abs()
    ddz = adz * (2 * d + 2.0 ** -16)[:, None]
    bad = {}

    def within(name, want, tol):
        if name not in got:
            return
        err = (got[name].double().reshape(want.shape) - want).abs()
        if not bool((err <= tol).all()):
            bad[name] = float((err / tol.clamp_min(1e-300)).max())
    within("loss", ref["loss"], ref["w"].abs() * 2 * ref["rest"] * (2 * d + 2.0 ** -18) + 2.0 ** -23 * ref["loss"].abs() + 1e-38)
    M = adz @ ref["A"]
    terms = 2.0 ** -11 * (2 if kind == "groups" else 1) if half else 2.0 ** -19
    E = ddz @ ref["A"] + 2.0 ** -38 * adz.amax(1)[:, None] * ref["A"].sum(0)[None]
    if kind == "matrix" and dtype == "bf16":
        terms, E = 2.0 ** -20, E + 2.0 ** -8 * ref["adz_others"] @ ref["A"]
    E = E + (terms + (V / 16 + 32) * 2.0 ** -22) * M
    want = ref["dz"] @ ref["W"]
    within("dx", want, E + step * (want.abs() + E) + tiny)
    within("dbias", ref["dz"].sum(0), (ddz + 2.0 ** -19 * adz).sum(0) + 1e-38)
    dzT = ref["dz"].t().contiguous()
    if kind == "rows":
        X, sx = ref["x"].sum(1, keepdim=True), head["s"]
        for name, f, mag in (("dscale", sx, head["smag"]), ("doffset", X.expand_as(sx), X.abs().expand_as(sx))):
            want = (ref["dz"] * f).sum(0)
            tol = (ddz * f.abs() + adz * 2.0 ** -19 * f.abs() + adz * 2.0 ** -22 * mag).sum(0)
            within(name, want, tol + 2.0 ** -23 * want.abs() + 1e-38)
        return bad
    M = adz.t().contiguous() @ ref["ax"]
    one = (ref["ax"] > 0).double().sum(0)[None]   # (x of +-1)
    E = (ddz.t().contiguous() @ ref["ax"] + ((2.0 ** -11 if kind == "matrix" and dtype == "bf16" else 2.0 ** -19) +
                                             (t / 16 + 32) * 2.0 ** -22) * M + 2.0 ** -38 * adz.amax(0)[:, None] * one)
    want = dzT @ ref["x"]
    if kind == "matrix":
        within("dweight", want, E + step * (want.abs() + E) + tiny)
        return bad
    e, G = head["e"], head["a"].shape[1]
    for name, ent in (("dscale", e), ("doffset", torch.ones_like(e))):
        def over_groups(v):
            return v.view(V, G, -1).sum(2)
        # (float32 sums of a group's columns, 64 at a time, joined in float64)
        tol = over_groups(E * ent.abs()) + 2.0 ** -19 * over_groups(M * ent.abs())
        value = over_groups(want * ent)
        within(name, value, tol + 2.0 ** -23 * value.abs() + 1e-38)
    return bad


def exact_inputs(m, t, dtype, cut, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randint(0, 2, (t, N), generator=gen, device="cuda") * 2 - 1).to(dtype_of(dtype))
    g = np.random.default_rng(seed)
    targets = g.integers(0, m, t).astype(np.int32)
    b = g.standard_normal(m).astype(np.float32)
    b[cut:] += np.log(m / (m - cut)).astype(np.float32)   # half of the mass behind the first piece's end
    w = (0.25 + g.random(t)).astype(np.float32)
    if t > 3:
        targets[::7] = -3
    return gen, x, dev(targets), dev(b), dev(w)


@pytest.mark.parametrize("kind,dtype,m,t", [("matrix", "bf16", 4200, 3), ("matrix", "fp16", 4200, 20), ("matrix", "fp32", 2100, 40),
                                           ("groups", "fp16", 2100, 150), ("groups", "bf16", 2100, 20), ("groups", "fp32", 2100, 10),
                                           ("rows", "bf16", 4200, 140), ("rows", "fp16", 4200, 20), ("rows", "fp32", 4200, 70)])
def test_longest_rows(kind, dtype, m, t):
    """Pieces of kept logits: 4096 rows of one plane, 2048 of two."""
    import torch
    import post_quantization_solver_amd as mpq
    cut = 2048 if kind == "groups" or (kind == "matrix" and dtype == "fp32") else 4096
    gen, x, targets, b, w = exact_inputs(m, t, dtype, cut, m + t)
    head = None
    if kind == "matrix":
        W = (torch.randint(-3, 4, (m, N), generator=gen, device="cuda") * 2.0 ** -8).to(dtype_of(dtype))
        got = mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w)
        ref = reference(x, dict(W=W), targets, b, w)
    else:
        # entries 0 .. 15 about 8; a a power of two, o a multiple of it: weights k 2^-8, |k| below 2^11, whose sums are
        # multiples of 2^-8 (rows: s', X and a s' + o' X as well)
        G = 16 if kind == "groups" else 1
        codes = torch.randint(5, 12, (m, N), generator=gen, device="cuda", dtype=torch.int32)
        a = torch.full((m, G), 2.0 ** -8, device="cuda")
        o = a * (torch.randint(-1, 2, (m, G), generator=gen, device="cuda") - 8).float()
        layer = mpq.pack_layer(codes, np.arange(16, dtype=np.float32)[:, None], a, o, group=N // 16 if G > 1 else None)
        got = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w)
        e, col = codes.double(), torch.arange(N, device="cuda") // (N // G)
        head = dict(e=e, a=a.double(), o=o.double(), mid=8.0, col=col)
        ref = reference(x, head, targets, b, w)
        if kind == "rows":
            X = ref["x"].sum(1, keepdim=True)
            middle = ref["x"] @ (e - 8.0).t().contiguous()
            head["s"] = middle + 8.0 * X
            head["smag"] = middle.abs() + 8.0 * X.abs()
            head["parts"] = (a.double()[:, 0] * middle).abs() + ((o + 8.0 * a).double()[:, 0] * X).abs()
    got = {k: v for k, v in got.items() if v is not None}
    assert not passes(got, ref, dtype, kind, b, head)
    # what has to fail: everything scaled, and each gradient without the last piece's rows
    assert set(passes({k: v.double() * 0.9 for k, v in got.items()}, ref, dtype, kind, b, head)) == set(got)
    short = ref["dz"][:, :cut] @ ref["W"][:cut]
    assert passes(dict(got, dx=short.to(x.dtype)), ref, dtype, kind, b, head).keys() == {"dx"}
    for k in got:
        if k not in ("loss", "dx"):
            part = got[k].clone()
            part[cut:] = 0
            assert passes(dict(got, **{k: part}), ref, dtype, kind, b, head).keys() == {k}


def test_addresses_past_32_bits():
    """Activations and their gradient of more than 2^31 elements: tokens from all over them."""
    import torch
    import post_quantization_solver_amd as mpq
    t, m = 33000, 96
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(t, N, dtype=torch.bfloat16, device="cuda")
    for k in range(0, t, 3300):
        x[k:k + 3300] = torch.randint(0, 2, (3300, N), generator=gen, device="cuda") * 2 - 1
    W = (torch.randint(-3, 4, (m, N), generator=gen, device="cuda") * 2.0 ** -8).to(torch.bfloat16)
    targets = torch.randint(m, (t,), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.ones(t, device="cuda")
    got = mpq.linear_cross_entropy(x, W, targets, need_dhead=False)
    for part in (slice(0, 40), slice(16368, 16408), slice(t - 40, t)):   # (the middle: about 2^30 elements; the end: past 2^31)
        ref = reference(x[part], dict(W=W), targets[part], None, w[part])
        own = dict(loss=got["loss"][part], dx=got["dx"][part])
        assert not passes(own, ref, "bf16", "matrix", None)
        assert passes(dict(own, dx=own["dx"] * 0.9), ref, "bf16", "matrix", None).keys() == {"dx"}
        assert passes(dict(own, dx=own["dx"].roll(1, 0)), ref, "bf16", "matrix", None).keys() == {"dx"}
