"""The cross entropy of a head and its gradients against the formulas in float64,
over codebooks, matrices, types, groups, sizes and strides.

Tolerances, with S_tv = sum |x a e'| + |o'| sum |x| + |b| the magnitudes that a logit
is the sum of (e' the entry less the middle level, o' the offset with it):
  - a logit: (n / 16 + 32) 2^-22 S for the float32 sums (as linear's), 2^-20 more
    where operands are two float16 terms (float32 x, weights of column groups);
    d_t the largest of a token's;
  - an exponential: 2^-23 (1 + |z - max|), weighted 2^-21 at most, its sums of 4096
    some 24 additions of 2^-24: 2^-18 in all.  The loss depends on R - z_r with the
    slope `rest` (1 less the target's probability): w rest (2 d_t + 2^-18), and one
    rounding; twice that covers the second order;
  - dz: relative 2 d_t + 2^-16 (|z - max| below 100);
  - dx: dz's, its terms and those of the weights of groups (2^-11 for one, 2^-20 for two;
    a bfloat16 matrix: dz in bfloat16, 2^-8, but for the target's, whose term is float32),
    elements below 2^-28 of the row's bound 2^-39 of it, float32 sums over the
    vocabulary (V / 16 + 32) 2^-22, one rounding of the result;
  - the head's gradients: dz's, s's own d_t, sums of 64 tokens (2^-19); of a matrix and
    of groups: dz^T's terms (2^-11 for a bfloat16 matrix, 2^-20), its elements below 2^-28
    of the largest dz's bound, float32 sums over the tokens and a group's columns.
"""
import numpy as np
import pytest

from parity_helpers import dev
from test_gpu_linear import STEP, dtype_of, make_layer, rows

pytestmark = pytest.mark.gpu


def reference(x, head, targets, bias, weights):
    """Loss, gradients and the magnitudes of the tolerances, float64 on the GPU.  head: dict(W) or dict(e, a, o, mid, col)."""
    import torch
    D = torch.float64
    x = x.double()
    t, n = x.shape
    skip = (targets < 0) | (weights == 0)
    x = torch.where(skip[:, None], torch.zeros((), dtype=D, device="cuda"), x)
    ax = x.abs()
    if "W" in head:
        W = head["W"].double()
        A = W.abs()
    else:
        col = head["col"]
        a, o = head["a"][:, col], head["o"][:, col]
        W = a * head["e"] + o
        A = (a * (head["e"] - head["mid"])).abs() + (o + a * head["mid"]).abs()
    b = torch.zeros(len(W), dtype=D, device="cuda") if bias is None else bias.double()
    z = x @ W.t().contiguous() + b
    S = ax @ A.t().contiguous() + torch.where(torch.isfinite(b), b.abs(), 0.0)
    r = targets.long().clamp(0, len(W) - 1)
    row = torch.arange(t, device="cuda")
    others = z.clone()
    others[row, r] = -np.inf
    R = torch.logsumexp(others, 1)
    gap = R - z[row, r]
    w = torch.where(skip, 0.0, weights.double())
    loss = w * torch.logaddexp(gap, torch.zeros_like(gap))
    rest = torch.sigmoid(gap)
    top = torch.maximum(R, z[row, r])
    lse = torch.logaddexp(R, z[row, r])
    dz = w[:, None] * torch.exp(z - lse[:, None])
    dz[row, r] = -w * rest
    dz[skip] = 0.0
    adz_others = dz.abs()
    adz_others[row, r] = 0.0
    return dict(x=x, ax=ax, W=W, A=A, z=z, S=S, loss=loss, rest=rest, w=w, dz=dz, skip=skip, top=top, adz_others=adz_others)


def check(got, ref, dtype, n, exact_terms, kind, head=None, need_dx=True, need_dhead=True):
    """exact_terms: the logits' operands are exact.  kind: "rows", "groups" or "matrix"."""
    import torch
    half = dtype != "fp32"
    V = len(ref["W"])
    t = len(ref["x"])
    step, tiny = STEP[dtype], 2.0 ** -25 if dtype == "fp16" else 1e-38
    d = ((n / 16 + 32) * 2.0 ** -22 + (0.0 if exact_terms else 2.0 ** -20)) * ref["S"].amax(1)
    rel = 2 * d + 2.0 ** -16

    def within(name, value, want, tol):
        err = (value.double() - want).abs()
        assert not torch.isnan(value).any(), name
        assert (err <= tol).all(), (name, float((err / tol.clamp_min(1e-300)).max()))
    within("loss", got["loss"], ref["loss"],
           ref["w"].abs() * 2 * ref["rest"] * (2 * d + 2.0 ** -18) + 2.0 ** -23 * ref["loss"].abs() + 1e-38)
    adz = ref["dz"].abs()
    ddz = adz * rel[:, None]
    bound = adz.amax(1)
    if need_dx:
        M, E = adz @ ref["A"], ddz @ ref["A"]
        terms = 2.0 ** -11 * (2 if kind == "groups" else 1) if half else 2.0 ** -19
        low = 2.0 ** -38 * (bound[:, None] * ref["A"].sum(0)[None] * (head["spread"] if head and "spread" in head else 1.0))
        if kind == "matrix" and dtype == "bf16":
            terms = 2.0 ** -20
            E = E + 2.0 ** -8 * ref["adz_others"] @ ref["A"]
        tol = E + terms * M + low + (V / 16 + 32) * 2.0 ** -22 * M
        within("dx", got["dx"], ref["dz"] @ ref["W"], tol + step * ((ref["dz"] @ ref["W"]).abs() + tol) + tiny)
    else:
        assert got["dx"] is None
    if not need_dhead:
        assert got["dbias"] is None
        return
    one = torch.ones(t, dtype=torch.float64, device="cuda")
    within("dbias", got["dbias"], ref["dz"].sum(0), (ddz + 2.0 ** -19 * adz).sum(0) + 1e-38)
    adzT, ddzT, dzT = adz.t().contiguous(), ddz.t().contiguous(), ref["dz"].t().contiguous()
    if kind == "matrix":
        M, E = adzT @ ref["ax"], ddzT @ ref["ax"]
        low = 2.0 ** -38 * bound.max() * (one @ ref["ax"])[None]
        tol = E + ((2.0 ** -11 if dtype == "bf16" else 2.0 ** -19) + (t / 16 + 32) * 2.0 ** -22) * M + low
        want = dzT @ ref["x"]
        within("dweight", got["dweight"], want, tol + step * (want.abs() + tol) + tiny)
        return
    e, mid, col, G = head["e"], head["mid"], head["col"], head["a"].shape[1]
    own = e - mid if kind == "rows" else e
    for name, ent, mag in (("dscale", e, own.abs() + (abs(mid) if kind == "rows" else 0.0)),
                           ("doffset", torch.ones_like(e), torch.ones_like(e))):
        if kind == "rows":
            s = ref["x"] @ ent.t().contiguous()
            m = ref["ax"] @ mag.t().contiguous()
            want = (ref["dz"] * s).sum(0)
            tol = ((ddz + adz * ((n / 16 + 32) * 2.0 ** -22 + 2.0 ** -19 + (0.0 if half else 2.0 ** -20))) * m).sum(0)
            within(name, got[name].reshape(-1), want, tol + 2.0 ** -23 * want.abs() + 1e-38)
        else:
            def over_groups(v):
                return torch.zeros(V, G, dtype=torch.float64, device="cuda").index_add_(1, col, v)
            want = over_groups((dzT @ ref["x"]) * ent)
            M = over_groups((adzT @ ref["ax"]) * mag)
            E = over_groups((ddzT @ ref["ax"]) * mag)
            low = 2.0 ** -38 * bound.max() * over_groups((one @ ref["ax"])[None] * mag)
            tol = E + (2.0 ** -19 + (t / 16 + 32) * 2.0 ** -22) * M + low
            within(name, got[name].reshape(V, G), want, tol + 2.0 ** -23 * want.abs() + 1e-38)


def inputs(g, m, n, t, dtype, bias, padded, pad, shift, weights=True):
    import torch
    x = rows(g, t, n, dtype, pad, shift)
    targets = g.integers(0, m, t).astype(np.int32)
    if padded:
        targets[g.random(t) < 0.3] = -1 - g.integers(0, 5)
    b = dev(g.standard_normal(m).astype(np.float32)) if bias else None
    w = (0.25 + g.random(t)).astype(np.float32) if weights else np.ones(t, np.float32)
    if padded and weights:
        w[g.random(t) < 0.2] = 0.0
    return x, dev(targets), b, dev(w)


def packed_case(name, m, n, t, dtype, group=0, offset=True, bias=True, padded=False, pad=0, shift=0, seed=0, scale_by=4.0,
                need_dx=True, need_dhead=True, workspace=None, spread=False):
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(500 + seed)
    codes, E, scale, off = make_layer(name, m, n, group, seed, offset)
    scale = (scale * scale_by / max(1.0, float(np.abs(E - E[len(E) // 2]).max()))).astype(np.float32)
    if spread:   # rows of very different scales
        scale = (scale * np.exp(2 * g.standard_normal(scale.shape))).astype(np.float32)
    if off is not None:
        off = (scale * g.standard_normal(scale.shape)).astype(np.float32) * 0.3
        if E.shape[1] == 1:
            off = off - scale * E[len(E) // 2, 0]
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off) if off is not None else None, group=group or None)
    x, targets, b, w = inputs(g, m, n, t, dtype, bias, padded, pad, shift)
    got = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w, need_dx=need_dx, need_dhead=need_dhead,
                                   workspace=workspace)
    d = E.shape[1]
    e = torch.from_numpy(np.asarray(E, np.float64)[codes].reshape(m, n)).cuda()
    G = -(-n // group) if 0 < group < n else 1
    mid = float(E[len(E) // 2, 0]) if d == 1 else 0.0
    col = torch.arange(n, device="cuda") // (group if G > 1 else n)
    a = layer.scale.double().reshape(m, G)
    o = layer.offset.double().reshape(m, G) if layer.offset is not None else torch.zeros_like(a)
    head = dict(e=e, a=a, o=o, mid=mid, col=col)
    if spread:
        # a row's dz times its scale against the largest scale: the bound's elements are that much smaller
        head["spread"] = float(a.max() / a.min())
    ref = reference(x, head, targets, b, w)
    check(got, ref, dtype, n, dtype != "fp32" and G == 1, "rows" if G == 1 else "groups", head, need_dx, need_dhead)
    return layer, x, targets, b, w, got


def matrix_case(m, n, t, dtype, bias=True, padded=False, pad=0, shift=0, seed=0, need_dx=True, need_dhead=True, size=4.0):
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(700 + seed)
    W = rows(g, m, n, dtype, pad, shift, scale=size / np.sqrt(n))
    x, targets, b, w = inputs(g, m, n, t, dtype, bias, padded, pad, shift)
    got = mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w, need_dx=need_dx, need_dhead=need_dhead)
    ref = reference(x, dict(W=W), targets, b, w)
    check(got, ref, dtype, n, dtype != "fp32", "matrix", None, need_dx, need_dhead)
    return W, x, targets, b, w, got


SHAPES = [(1, 1, 1), (2, 8, 1), (17, 72, 3), (64, 64, 64), (65, 136, 65), (300, 128, 33), (1000, 264, 130), (4099, 64, 17),
          (5000, 520, 260)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,n,t", SHAPES)
def test_matrix_sizes(dtype, m, n, t):
    matrix_case(m, n, t, dtype, seed=m + t, padded=t > 3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,n,t", SHAPES)
def test_packed_sizes(dtype, m, n, t):
    packed_case("e8240" if n % 8 == 0 and m % 2 else "s16", m, n, t, dtype, seed=m + t, padded=t > 3)


@pytest.mark.parametrize("name", ["s2", "s3", "s8", "s16", "s17", "s64", "levels", "vec", "e865536", "e81", "e8240", "e8241",
                                  "e830000"])
@pytest.mark.parametrize("t", [2, 150])
@pytest.mark.parametrize("offset", [False, True])
def test_packed_books(name, t, offset):
    packed_case(name, 333, 264, t, "bf16", seed=t + len(name), offset=offset or name[0] == "s")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,n,group", [("s16", 512, 128), ("s16", 500, 128), ("s64", 320, 64), ("s16", 200, 33),
                                          ("s8", 96, 1), ("s16", 256, 256), ("s16", 100, 4096)])
@pytest.mark.parametrize("t", [1, 20, 140])
def test_packed_groups(dtype, name, n, group, t):
    packed_case(name, 210, n, t, dtype, group=group, seed=n + t, padded=t > 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,n,group", [("s3", 256, 0), ("s16", 500, 0), ("s16", 1152, 128), ("s64", 333, 0), ("s64", 320, 64),
                                          ("levels", 130, 0), ("vec", 264, 0), ("e8240", 520, 0), ("e865536", 1096, 0)])
@pytest.mark.parametrize("t", [1, 2, 3, 4, 5])
def test_few_tokens(dtype, name, n, group, t):
    """The gradients of some tokens, straight from the codes or through planes; rows behind a last whole tile."""
    packed_case(name, 1003, n, t, dtype, group=group, seed=n + t, padded=t == 4)


@pytest.mark.parametrize("t", [1, 3])
@pytest.mark.parametrize("name", ["s16", "e8240"])
def test_few_tokens_wanted_outputs(name, t):
    """The parts alone are the bits of the whole here too; a long vocabulary, many splits of its rows."""
    import torch
    import post_quantization_solver_amd as mpq
    head, x, targets, b, w, full = packed_case(name, 20011, 64, t, "bf16", seed=t)
    for need_dx, need_dhead in ((False, False), (True, False), (False, True)):
        got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dx=need_dx, need_dhead=need_dhead)
        for k, v in got.items():
            assert v is None or torch.equal(v, full[k]), k


@pytest.mark.parametrize("name,group", [("s16", 0), ("s16", 128), ("s64", 0), ("e8240", 0), ("vec", 0)])
def test_few_tokens_that_are_not_read(name, group):
    """Of four tokens: one without a target and NaN in its row, one of weight 0 with infinities, one past the vocabulary;
    a vocabulary with rows masked by -inf; a workspace that held something else."""
    import torch
    import post_quantization_solver_amd as mpq
    head, x, targets, b, w, _ = packed_case(name, 700, 256, 4, "bf16", group=group, seed=8)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    b[::3] = -float("inf")
    targets.copy_(torch.tensor([4, 5, 7, 10], dtype=torch.int32))
    alone = [mpq.linear_cross_entropy(x[k:k + 1], head, targets[k:k + 1], bias=b, weights=w[k:k + 1]) for k in range(4)]
    targets[0], w[1] = -1, 0.0
    x[0], x[1] = float("nan"), float("inf")
    got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, workspace=ws)
    assert not got["loss"][:2].any() and not got["dx"][:2].any()
    for k in (2, 3):   # (sums of another split: dx is rounded to bfloat16, 2^-8 of a value near the row's largest at most)
        assert torch.isfinite(got["loss"][k]) and (got["loss"][k] - alone[k]["loss"][0]).abs() <= 2.0 ** -18 * got["loss"][k].abs()
        one = alone[k]["dx"][0].float()
        assert ((got["dx"][k].float() - one).abs() <= 2.0 ** -7 * one.abs() + 2.0 ** -14 * one.abs().max()).all()
    assert not got["dbias"][::3].any()
    total = alone[2]["dbias"].double() + alone[3]["dbias"].double()
    assert ((got["dbias"].double() - total).abs() <= 2.0 ** -17 * (alone[2]["dbias"].abs() + alone[3]["dbias"].abs())).all()
    targets[2] = 700
    got2 = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, workspace=ws)
    assert torch.isnan(got2["loss"][2]) and torch.isnan(got2["dx"][2]).all()
    assert torch.equal(got2["loss"][3], got["loss"][3]) and torch.equal(got2["dx"][3], got["dx"][3])
    assert not got2["dx"][:2].any()


@pytest.mark.parametrize("n", [512, 500])
@pytest.mark.parametrize("t", [1, 3, 70])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_matrix_gradient_is_rounded_once(dtype, t, n):
    """The gradient of a matrix is as near as its type allows: by their mean square relative to the gradient, errors are
    those of rounding the formula's value (a second rounding of 11 bits before it would make float16's 1.41 of that; dz
    in float32 is good to some 2^-18).  A bfloat16 matrix has dz in one term: each product dz x is off by 2^-11 of itself
    at most, so an element by 2^-11 sum |dz| |x|, which is more than its own rounding where the tokens cancel."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(40 + t)
    W = rows(g, 600, n, dtype, 0, 0, scale=1.0 / np.sqrt(n))
    x, targets, b, w = inputs(g, 600, n, t, dtype, False, False, 0, 0)
    got = mpq.linear_cross_entropy(x, W, targets, weights=w)["dweight"]
    ref = reference(x, dict(W=W), targets, None, w)
    want = ref["dz"].t().contiguous() @ ref["x"]
    # (float16's subnormal steps say nothing of this)
    keep = want.abs() > (2.0 ** -12 if dtype == "fp16" else 0.0)
    assert keep.sum() > 500

    def size(v):
        return float((v[keep] / want.abs()[keep].clamp_min(1e-3 * float(want.abs().mean()))).square().mean().sqrt())
    terms = 2.0 ** -11 * size(ref["dz"].abs().t().contiguous() @ ref["ax"]) if dtype == "bf16" else 0.0
    assert size(got.double() - want) <= 1.2 * size(want.to(got.dtype).double() - want) + terms + (2.0 ** -16 if dtype == "fp32" else 0.0)


def test_a_column_a_group():
    """As many groups as columns: more than a grid can sum up in one piece."""
    import torch
    import post_quantization_solver_amd as mpq
    m, n, t = 33000, 2048, 3
    gen = torch.Generator(device="cuda").manual_seed(7)
    codes = torch.randint(16, (m, n), generator=gen, device="cuda", dtype=torch.int32)
    E = np.arange(16, dtype=np.float64)[:, None] - 7.5
    a = torch.rand(m, n, generator=gen, device="cuda") * 0.01 + 0.005
    o = torch.randn(m, n, generator=gen, device="cuda") * 0.01
    layer = mpq.pack_layer(codes, E, a, o, group=1)
    x, targets, b, w = inputs(np.random.default_rng(7), m, n, t, "bf16", True, False, 0, 0)
    got = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w)
    head = dict(e=codes.double() - 7.5, a=a.double(), o=o.double(), mid=0.5, col=torch.arange(n, device="cuda"))
    check(got, reference(x, head, targets, b, w), "bf16", n, False, "groups", head)


def test_addresses_past_32_bits():
    """Activations and their gradient of more than 2^31 elements: the first and the last tokens."""
    import torch
    import post_quantization_solver_amd as mpq
    t, n, m = 33000, 65536, 96
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    for k in range(0, t, 3300):
        x[k:k + 3300] = torch.randn(3300, n, generator=gen, device="cuda")
    W = (torch.randn(m, n, generator=gen, device="cuda") * (3.0 / 256)).to(torch.bfloat16)
    targets = torch.randint(m, (t,), generator=gen, device="cuda", dtype=torch.int32)
    w = torch.ones(t, device="cuda")
    got = mpq.linear_cross_entropy(x, W, targets, need_dhead=False)
    for part in (slice(0, 40), slice(t - 40, t)):
        ref = reference(x[part], dict(W=W), targets[part], None, w[part])
        check(dict(loss=got["loss"][part], dx=got["dx"][part], dbias=None), ref, "bf16", n, True, "matrix", need_dhead=False)


@pytest.mark.parametrize("need_dx,need_dhead", [(False, False), (True, False), (False, True)])
def test_wanted_outputs(need_dx, need_dhead):
    """The parts alone are the bits of the whole."""
    import torch
    import post_quantization_solver_amd as mpq
    for make, kw in ((packed_case, dict(name="s16", group=0)), (packed_case, dict(name="s16", group=64)),
                     (packed_case, dict(name="e8240")), (matrix_case, {})):
        head, x, targets, b, w, full = make(m=700, n=256, t=100, dtype="bf16", seed=3, **kw)
        got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dx=need_dx, need_dhead=need_dhead)
        for k, v in got.items():
            wanted = k == "loss" or (need_dx if k == "dx" else need_dhead)
            assert (v is not None) == wanted
            if wanted:
                assert torch.equal(v, full[k]), k


@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (3, 1), (0, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides(pad, shift, dtype):
    matrix_case(130, 72, 70, dtype, pad=pad, shift=shift, seed=pad)
    packed_case("s16", 130, 72, 70, dtype, pad=pad, shift=shift, seed=pad)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pieces(dtype):
    """Vocabularies of several pieces: many tokens, and long rows."""
    matrix_case(2600, 40, 33000, dtype, padded=True, seed=1)
    packed_case("s16", 2600, 40, 33000, dtype, padded=True, seed=2)
    packed_case("s64", 2060, 72, 33001, dtype, padded=True, seed=2)
    packed_case("s16", 2100, 192, 33000, dtype, group=64, seed=3)
    packed_case("s16", 2100, 96, 33000, dtype, group=32, seed=3)
    packed_case("e8240", 2300, 40, 33000, dtype, seed=4, offset=False)
    packed_case("s16", 2500, 8192, 5, dtype, seed=5)
    matrix_case(2600, 128, 33000, dtype, padded=True, seed=7)
    matrix_case(2570, 64, 33000, dtype, pad=1, seed=9)


@pytest.mark.parametrize("kind,dtype,m,t", [("matrix", "bf16", 4200, 3), ("matrix", "fp32", 2100, 40), ("groups", "fp16", 2100, 150),
                                           ("rows", "bf16", 4200, 140)])
def test_pieces_of_kept_logits(kind, dtype, m, t):
    """The longest rows: the planes of a few thousand of them are pieces, their logits are kept."""
    import torch
    import post_quantization_solver_amd as mpq
    n = 65536
    gen = torch.Generator(device="cuda").manual_seed(m + t)
    g = np.random.default_rng(m + t)
    x, targets, b, w = inputs(g, m, n, t, dtype, True, True, 0, 0)
    if kind == "matrix":
        W = (torch.randn(m, n, generator=gen, device="cuda") * (3.0 / 256)).to(dtype_of(dtype))
        got = mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w)
        ref = reference(x, dict(W=W), targets, b, w)
        check(got, ref, dtype, n, dtype != "fp32", "matrix")
        return
    E = np.arange(16, dtype=np.float32)[:, None]
    codes = torch.randint(0, 16, (m, n), generator=gen, device="cuda", dtype=torch.int32)
    group = 4096 if kind == "groups" else 0
    G = n // group if group else 1
    a = (0.5 + torch.rand(m, G, generator=gen, device="cuda")) * (3.0 / 256 / 4.6)
    o = a * (torch.randn(m, G, generator=gen, device="cuda") * 0.3 - 8.0)
    layer = mpq.pack_layer(codes, E, a, o, group=group or None)
    got = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w)
    col = torch.arange(n, device="cuda") // (group or n)
    head = dict(e=codes.double(), a=a.double(), o=o.double(), mid=8.0, col=col)
    ref = reference(x, head, targets, b, w)
    check(got, ref, dtype, n, group == 0, kind, head)


def test_rows_of_very_different_scales():
    packed_case("s16", 1000, 256, 100, "bf16", spread=True, seed=9)
    packed_case("e8240", 1000, 256, 100, "fp32", spread=True, seed=9)


@pytest.mark.parametrize("book", ["matrix", "s16", "e8240"])
def test_certain_tokens(book):
    """Targets that are all but certain: small losses and gradients keep their relative accuracy."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(4)
    m, n, t = 500, 128, 64
    x, targets, _, w = inputs(g, m, n, t, "fp32", False, False, 0, 0)
    bias = np.zeros(m, np.float32)
    targets[:] = 7
    bias[7] = 30.0   # rest some e^-30 of the others' mass
    b = dev(bias)
    if book == "matrix":
        head = rows(g, m, n, "fp32", scale=0.3 / np.sqrt(n))
        ref = reference(x, dict(W=head), targets, b, w)
    else:
        head, *_ = packed_case(book, m, n, t, "fp32", seed=8, offset=False)
        head.scale.mul_(0.05)
        lay = make_layer(book, m, n, 0, 8, False)
        e = torch.from_numpy(np.asarray(lay[1], np.float64)[lay[0]].reshape(m, n)).cuda()
        mid = float(lay[1][len(lay[1]) // 2, 0]) if lay[1].shape[1] == 1 else 0.0
        a = head.scale.double().reshape(m, 1)
        hd = dict(e=e, a=a, o=torch.zeros_like(a), mid=mid, col=torch.zeros(n, dtype=torch.long, device="cuda"))
        ref = reference(x, hd, targets, b, w)
    got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    assert float(ref["loss"].max()) < 1e-6
    check(got, ref, "fp32", n, False, "matrix" if book == "matrix" else "rows", None if book == "matrix" else hd)


def test_masked_vocabulary():
    """Biases of -inf: out of the vocabulary; as a target +inf; a vocabulary without any; a row of one token."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(5)
    m, n, t = 300, 64, 40
    W = rows(g, m, n, "fp32", scale=0.3)
    x, targets, _, w = inputs(g, m, n, t, "fp32", False, False, 0, 0)
    b = torch.zeros(m, device="cuda")
    b[::3] = -np.inf
    targets = (targets // 3 * 3 + 1).clamp_max(m - 1).int()
    ref = reference(x, dict(W=W), targets, b, w)
    check(mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w), ref, "fp32", n, False, "matrix")
    # a masked target
    hidden = targets.clone()
    hidden[5] = 3
    r = mpq.linear_cross_entropy(x, W, hidden, bias=b, weights=w)
    assert torch.isposinf(r["loss"][5]) and int(torch.isinf(r["loss"]).sum()) == 1
    assert all(torch.isfinite(r[k]).all() for k in ("dx", "dweight", "dbias"))
    assert float((r["dbias"].sum()).abs()) < 1e-4      # every token's dz adds up to nothing
    # nobody left
    r = mpq.linear_cross_entropy(x, W, targets, bias=torch.full((m,), -np.inf, device="cuda"), weights=w)
    assert torch.isposinf(r["loss"]).all() and not any(r[k].any() for k in ("dx", "dweight", "dbias"))
    # one token left
    b = torch.full((m,), -np.inf, device="cuda")
    b[11] = 0.5
    r = mpq.linear_cross_entropy(x, W, torch.full_like(targets, 11), bias=b, weights=w)
    assert not any(v.any() for v in r.values())


@pytest.mark.parametrize("kind", ["rows", "groups", "matrix"])
def test_rows_that_are_not_read(kind):
    """Padding and weight 0 with NaN and infinities in x: zeros, and the other rows as if they were not there."""
    import torch
    import post_quantization_solver_amd as mpq
    case = dict(rows=dict(name="s16"), groups=dict(name="s16", group=64), matrix={})[kind]
    make = matrix_case if kind == "matrix" else packed_case
    head, x, targets, b, w, _ = make(m=400, n=128, t=90, dtype="bf16", seed=6, **case)
    targets[10:20] = -1
    w[30:40] = 0.0
    x[10:20], x[30:40] = 0.0, 0.0
    clean = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    x[10:15], x[15:20], x[30:40] = float("nan"), float("inf"), -float("inf")
    got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    for k in got:
        assert torch.equal(got[k], clean[k]), k
    gone = torch.zeros(90, dtype=torch.bool, device="cuda")
    gone[10:20] = gone[30:40] = True
    assert not got["loss"][gone].any() and not got["dx"][gone].any()
    # one row is NaN: its own loss and dx, not the others'
    x[50] = float("nan")
    r = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dhead=False)
    live = torch.arange(90, device="cuda") != 50
    assert torch.isnan(r["loss"][50]) and torch.isnan(r["dx"][50]).all()
    assert torch.equal(r["loss"][live], got["loss"][live]) and torch.equal(r["dx"][live], got["dx"][live])
    # a target past the vocabulary
    x[50] = 1.0
    targets[50] = 400
    r = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    assert torch.isnan(r["loss"][50]) and torch.isnan(r["dx"][50]).all() and torch.isnan(r["dbias"]).all()
    assert torch.equal(r["loss"][live], got["loss"][live]) and torch.equal(r["dx"][live], got["dx"][live])


def test_no_tokens_and_no_live_tokens():
    import torch
    import post_quantization_solver_amd as mpq
    for make, kw in ((packed_case, dict(name="s16", group=32)), (packed_case, dict(name="e8240")), (matrix_case, {})):
        head, x, targets, b, w, full = make(m=70, n=96, t=5, dtype="bf16", seed=1, **kw)
        r = mpq.linear_cross_entropy(x[:0], head, targets[:0], bias=b)
        assert r["loss"].shape == (0,) and r["dx"].shape == (0, 96)
        assert not any(v.any() for v in r.values()) and all(r[k].shape == full[k].shape for k in r if k[0] == "d" and k != "dx")
        r = mpq.linear_cross_entropy(x, head, torch.full_like(targets, -1), bias=b)
        assert not any(v.any() for v in r.values())


def test_against_differences():
    """The gradients against central differences of the loss, in float64 of the formula's own inputs.

    Steps of 1e-3 of float32 losses of some 5 (error 2^-20): differences are good to 2^-20 5 / 1e-3 and the second
    order's 1e-6 of the third derivative (below 30): 6e-3 in all."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(12)
    codes, E, scale, off = make_layer("s16", 50, 64, 0, 12)
    scale, off = dev(scale * 0.3), dev(off * 0.3)
    layer = mpq.pack_layer(dev(codes), E, scale, off)
    x, targets, b, w = inputs(g, 50, 64, 6, "fp32", True, False, 0, 0)
    got = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w)

    def total():
        return float(mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w, need_dx=False, need_dhead=False)["loss"]
                     .double().sum())
    for tensor, name in ((x, "dx"), (b, "dbias"), (scale, "dscale"), (off, "doffset")):
        flat, grad = tensor.view(-1), got[name].reshape(-1)
        for k in g.integers(0, flat.numel(), 6):
            old, h = float(flat[k]), 1e-3 if name != "dscale" else 1e-4
            flat[k] = old + h
            up, hi = total(), float(flat[k])
            flat[k] = old - h
            down, lo = total(), float(flat[k])
            flat[k] = old
            assert abs((up - down) / (hi - lo) - float(grad[k])) <= 6e-3 * (1 if name != "dscale" else 20), (name, k)


def test_repeatable_shared_workspace_other_stream():
    """The same bits again, from a workspace that held something else, and on another stream than the current one."""
    import torch
    import post_quantization_solver_amd as mpq
    ws = torch.full((600 << 20,), 255, dtype=torch.uint8, device="cuda")
    for make, kw in ((packed_case, dict(name="s16", group=64)), (packed_case, dict(name="e865536")), (matrix_case, {})):
        head, x, targets, b, w, first = make(m=1500, n=512, t=200, dtype="bf16", seed=2, padded=True, **kw)
        again = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, workspace=ws)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], again[k]) and torch.equal(first[k], other[k]), k


def test_captured_with_the_step():
    """A head's loss and the step of its scales captured as one graph: replays against eager calls, eager work between."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(3)
    made = []
    for _ in range(2):
        codes, E, scale, off = make_layer("s16", 600, 256, 64, 3)
        layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=64)
        made.append((layer, mpq.AdamW([layer.scale, layer.offset], lr=1e-4, state_bits=8, seed=1)))
    x, targets, b, w = inputs(g, 600, 256, 100, "bf16", True, True, 0, 0)

    def tune(layer, opt):
        r = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w)
        norm = opt.step([r["dscale"], r["doffset"]], max_norm=1.0)
        return r["loss"], norm
    tune(*made[0])
    tune(*made[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            loss, norm = tune(*made[0])
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        x.mul_(0.9)
        graph.replay()
        want, want_norm = tune(*made[1])
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and torch.equal(norm, want_norm)
        assert torch.equal(made[0][0].scale, made[1][0].scale) and torch.equal(made[0][0].offset, made[1][0].offset)
        (x.float() @ x.float().t()).sum().item()
    assert int(made[0][1].steps) == 5


def test_refusals():
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(1)
    codes, E, scale, off = make_layer("s16", 50, 64, 0, 1)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off))
    W = rows(g, 50, 64, "fp32")
    x = rows(g, 4, 64, "fp32")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    call = mpq.linear_cross_entropy
    for bad in (lambda: call(x.cpu(), layer, tok), lambda: call(x.double(), layer, tok), lambda: call(x, W.half(), tok),
                lambda: call(x, W, tok.long()), lambda: call(x, W, tok.cpu()), lambda: call(x, W, tok, bias=W[0]),
                lambda: call(x, W, tok, weights=W[0]), lambda: call(x, W, tok, bias=torch.zeros(50, device="cuda").half()),
                lambda: call(x[:, :63], W, tok), lambda: call(x[:, :63], layer, tok), lambda: call(x, W.t(), tok),
                lambda: call(x, W[:0], tok), lambda: call(x, W, tok[:3]), lambda: call(x, None, tok)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(mpq.MPQError):
        call(x, W, tok, workspace=torch.empty(1000, dtype=torch.uint8, device="cuda"))
