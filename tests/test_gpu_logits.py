"""Token log probabilities and distillation against float64, at the sizes,
strides and masks where they can go wrong.

Tolerances.  One exponential is off by a unit in its last place, 2^-23, its
argument y by three half units (a difference, a factor, a product), 3 2^-24 |y|
ln 2 relative; weighted by 2^y the mean of |y| is at most log2 V <= 20 (no sum
has a larger one), eight terms are summed in three roundings of 2^-24: the sum
is off by (2 + 3 + 42) 2^-24, under 2^-18, and so is a log of it.  An output is rounded to float32: 2^-24 |value|.
The entropy's mean of y carries a relative 2^-18 of at most 20.  A gradient is
weight / T (q - p) with q off by 2^-18 and by 3 2^-24 |y| (|y| < 64 where q
matters: 2^-17), p by 2^-24, then one rounding to its type, half a step.
"""
import numpy as np
import pytest

from oracle import ops_oracle as R
from parity_helpers import dev, host

pytestmark = pytest.mark.gpu

STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def rows(g, t, V, dtype, spread=3.0, pad=0, shift=0):
    """t x V logits as a view with row stride V + pad starting `shift` elements into its buffer."""
    import torch
    buf = torch.from_numpy((g.standard_normal(t * (V + pad) + shift + 8) * spread).astype(np.float32)).cuda()
    buf = buf.to(dtype_of(dtype))
    return torch.as_strided(buf, (t, V), (V + pad, 1), shift)


def check_logprobs(z, tokens, top):
    import torch
    import post_quantization_solver_amd as mpq
    r = mpq.token_logprobs(z, dev(tokens), top=top)
    torch.cuda.synchronize()
    ref = R.token_logprobs(z.double().cpu().numpy(), tokens, top)
    for k in ("lse", "logprob", "entropy") + (("top_logprobs",) if top else ()):
        got, want = host(r[k]).astype(np.float64), ref[k]
        fin = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), fin) and np.array_equal(np.isnan(got), np.isnan(want)), k
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)]), k
        tol = 2.0 ** -24 * np.abs(want[fin]) + 2.0 ** -18 * (20 if k == "entropy" else 1)
        err = np.abs(got[fin] - want[fin])
        assert (err <= tol).all(), (k, err.max(), tol.min())
    if top:
        assert np.array_equal(host(r["top_ids"]), ref["top_ids"])
    return r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,V,top", [(1, 1, 1), (3, 2, 4), (2, 63, 5), (5, 1000, 20), (2, 4097, 128), (1, 32000, 20),
                                     (7, 16385, 64), (3, 50257, 1), (600, 8192, 0), (2, 131071, 100)])
def test_logprobs(dtype, t, V, top):
    g = np.random.default_rng(V + t)
    z = rows(g, t, V, dtype)
    tokens = g.integers(-1, V, t).astype(np.int32)
    check_logprobs(z, tokens, top)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(3, 1), (8, 0), (0, 5)])
def test_logprobs_strides(dtype, pad, shift):
    g = np.random.default_rng(pad * 10 + shift)
    z = rows(g, 4, 9001, dtype, pad=pad, shift=shift)
    check_logprobs(z, g.integers(0, 9001, 4).astype(np.int32), 33)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_masks_and_ties(dtype):
    import torch
    g = np.random.default_rng(5)
    V = 20000
    z = rows(g, 12, V, dtype).clone()
    z[0] = float("-inf")                    # nothing left
    z[1] = float("-inf")
    z[1, 17] = 2.5                          # one alternative
    z[2, : V - 3] = float("-inf")           # three
    z[3] = 0.25                             # all equal: more than fit the candidates
    z[4] = torch.round(z[4])                # many ties
    z[5, 777] = float("nan")
    z[6, 777] = float("inf")
    z[7] = torch.finfo(z.dtype).min         # masked by the type's lowest value
    z[7, 5:9] = 1.0
    z[8, ::2] = float("-inf")
    z[9] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0).to(z.dtype)   # zeros of both signs tie
    z[10] = torch.arange(V, device="cuda").float().to(z.dtype) / V
    tokens = np.array([3, 17, 4, 9, 2, 777, -1, 6, 1, 0, V - 1, V], np.int32)
    check_logprobs(z, tokens, 128)


def test_logprobs_without_tokens_and_empty():
    import torch
    import post_quantization_solver_amd as mpq
    z = torch.randn(3, 100, device="cuda")
    r = mpq.token_logprobs(z)
    assert r["logprob"] is None and r["top_ids"] is None and r["lse"].shape == (3,)
    r = mpq.token_logprobs(z[:0], torch.empty(0, dtype=torch.int32, device="cuda"), top=4)
    assert r["lse"].shape == (0,) and r["top_ids"].shape == (0, 4)


def teacher_list(g, z, k, noise=0.3):
    """A teacher near the student: its top k and their log probabilities."""
    a = z.double().cpu().numpy() + noise * g.standard_normal(z.shape)
    lp = a - np.log(np.exp(a - a.max(1, keepdims=True)).sum(1, keepdims=True)) - a.max(1, keepdims=True)
    ids = np.argsort(-lp, axis=1, kind="stable")[:, :k]
    return ids.astype(np.int32), np.take_along_axis(lp, ids, 1).astype(np.float32)


def check_distill(z, ids, teacher, dtype, T=1.0, tail=False, weights=None):
    import torch
    import post_quantization_solver_amd as mpq
    ref_z = z.double().cpu().numpy()
    loss, grad, scale = R.distill(ref_z, ids, teacher.astype(np.float64), T, tail, weights)
    w = None if weights is None else dev(weights.astype(np.float32))
    r = mpq.distill(z, dev(ids), dev(teacher), temperature=T, tail=tail, weights=w)
    torch.cuda.synchronize()
    wt = np.ones(z.shape[0]) if weights is None else weights
    got = host(r["loss"]).astype(np.float64)
    assert (np.abs(got - loss) <= 2.0 ** -24 * np.abs(loss) + 2.0 ** -17 * np.abs(wt)).all(), np.abs(got - loss).max()
    g = r["grad"].double().cpu().numpy()
    tol = STEP[dtype] * np.abs(grad) + 2.0 ** -16 * np.abs(scale) + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    assert (np.abs(g - grad) <= tol).all(), (np.abs(g - grad) / tol).max()
    # the loss alone, and the gradient written over the logits
    alone = mpq.distill(z, dev(ids), dev(teacher), temperature=T, tail=tail, weights=w, grad=False)
    assert alone["grad"] is None and torch.equal(alone["loss"], r["loss"])
    zc = z.clone()
    over = mpq.distill(zc, dev(ids), dev(teacher), temperature=T, tail=tail, weights=w, grad=zc)
    assert over["grad"] is zc and torch.equal(zc, r["grad"]) and torch.equal(over["loss"], r["loss"])
    return r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("t,V,k,T,tail", [(1, 3, 2, 1.0, False), (4, 100, 100, 1.0, True), (3, 1000, 5, 2.0, False),
                                          (2, 50257, 100, 4.0, False), (5, 16385, 64, 1.0, True), (1, 128, 128, 1.0, False),
                                          (300, 4096, 20, 1.0, True), (2, 70001, 1, 1.0, True), (3, 999, 0, 1.0, True)])
def test_distill(dtype, t, V, k, T, tail):
    g = np.random.default_rng(V + k)
    z = rows(g, t, V, dtype, spread=2.5, pad=5, shift=1)
    ids, lp = teacher_list(g, z, k)
    check_distill(z, ids, lp, dtype, T, tail)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_lists(tail):
    """Entries outside the vocabulary, tokens listed twice, masses of zero, empty lists, weights."""
    g = np.random.default_rng(8)
    V, k = 9000, 12
    z = rows(g, 6, V, "fp32", spread=2.0)
    ids, lp = teacher_list(g, z, k)
    ids[0, 3:6] = [-1, V, 2 ** 31 - 1]
    ids[1, 5] = ids[1, 2]
    ids[1, 7] = ids[1, 2]
    lp[2, 4] = -np.inf
    ids[3] = -1
    weights = np.array([0.5, 2.0, 1.0, 3.0, 0.0, 1.0])
    z = z.clone()
    z[4] = float("nan")     # weight 0: not read
    check_distill(z, ids, lp, "fp32", 1.0, tail, weights)


def test_distill_masked_tail():
    """A student whose unlisted tokens are masked: an infinite loss where the teacher has mass there, and none
    where it has not."""
    import torch
    import post_quantization_solver_amd as mpq
    z = torch.full((2, 64), float("-inf"), device="cuda")
    z[:, :2] = 0.0
    ids = torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device="cuda")
    lp = torch.tensor([[-1.0, -2.0], [-0.6931472, -0.6931472]], device="cuda")
    r = mpq.distill(z, ids, lp, tail=True)
    loss = host(r["loss"])
    assert np.isposinf(loss[0]) and abs(loss[1]) < 1e-6
    assert np.abs(host(r["grad"])[1]).max() < 1e-6


def test_distill_gradient_differences():
    """The gradient against differences of the loss in float64 arithmetic over float32 losses."""
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(3)
    z = rows(g, 1, 40, "fp32", spread=1.0).clone()
    ids, lp = teacher_list(g, z, 7, noise=1.0)
    for tail in (False, True):
        grad = host(mpq.distill(z, dev(ids), dev(lp), tail=tail)["grad"])[0]
        h = 2.0 ** -6
        for j in (0, int(ids[0, 0]), int(ids[0, 6]), 39):
            up, dn = z.clone(), z.clone()
            up[0, j] += h
            dn[0, j] -= h
            fu, fd = (float(mpq.distill(v, dev(ids), dev(lp), tail=tail, grad=False)["loss"]) for v in (up, dn))
            # central differences: the third derivative of a softmax loss is below 1; the losses carry 2^-18
            assert abs((fu - fd) / (2 * h) - grad[j]) <= h * h / 6 + 2.0 ** -18 / h


def test_teacher_list_to_distill():
    """token_logprobs' list of one model as the teacher of another, on a side stream."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(4)
    teacher = rows(g, 16, 32001, "bf16")
    student = (teacher.float() + 0.2 * torch.randn_like(teacher.float())).bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        top = mpq.token_logprobs(teacher, top=64)
        r = mpq.distill(student, top["top_ids"], top["top_logprobs"], tail=True)
    torch.cuda.current_stream().wait_stream(side)
    loss, grad, _ = R.distill(student.double().cpu().numpy(), host(top["top_ids"]),
                              host(top["top_logprobs"]).astype(np.float64), tail=True)
    assert np.abs(host(r["loss"]) - loss).max() < 2.0 ** -17
    same = mpq.distill(teacher, top["top_ids"], top["top_logprobs"], tail=True)
    assert np.abs(host(same["loss"])).max() < 2.0 ** -17   # a teacher has nothing to learn from itself


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,k", [(16, 1), (16, 64), (130, 1), (130, 64)])
def test_divergences_near_zero(dtype, t, k):
    """A student that is nearly the teacher.  The listed elements enter in float64 and the unlisted sum with a relative
    error of at most 2^-20 (float32's rounding of an exponent of up to 2^5 and of its power), which the loss has times
    the difference of the two remainders; 2^-23 of the loss is its own rounding, and 2^-36 the series'.  log2(e) is
    used as a float32, half a step of 2^-23 off at most: logits times 1 + 2^-24 / 1.44, which the loss, whose slope in
    that factor is sum_j (q_j - p_j) z_j (unlisted p_j = q_j pt / qt), has 2^-24 times."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(31 + t + k)
    teacher = rows(g, t, 20011, "fp32").double().cpu().numpy() * 2
    lp = teacher - np.log(np.exp(teacher - teacher.max(1, keepdims=True)).sum(1, keepdims=True)) - teacher.max(1, keepdims=True)
    ids = np.argsort(-lp, axis=1)[:, :k].astype(np.int32)
    lists = np.take_along_axis(lp, ids.astype(np.int64), 1).astype(np.float32)
    student = torch.from_numpy(teacher + 0.01 * g.standard_normal(teacher.shape)).to("cuda", dtype_of(dtype))
    got = mpq.distill(student, dev(ids), dev(lists), tail=True)["loss"].double().cpu().numpy()
    z = student.double().cpu().numpy()
    z = z - z.max(1, keepdims=True)
    lq = z - np.log(np.exp(z).sum(1, keepdims=True))
    p = np.exp(lists.astype(np.float64))
    hidden = np.ones(z.shape, bool)
    np.put_along_axis(hidden, ids.astype(np.int64), False, 1)
    pt, qt = 1 - p.sum(1), np.where(hidden, np.exp(lq), 0).sum(1)
    want = (p * (lists - np.take_along_axis(lq, ids.astype(np.int64), 1))).sum(1) + pt * (np.log(pt) - np.log(qt))
    full = np.exp(lq) * (pt / qt)[:, None]
    np.put_along_axis(full, ids.astype(np.int64), p, 1)
    slope = (np.abs(np.exp(lq) - full) * np.abs(z)).sum(1)
    tol = 2.0 ** -20 * np.abs(pt - qt) + 2.0 ** -24 * slope + 2.0 ** -23 * np.abs(want) + 2.0 ** -36
    assert (np.abs(got - want) <= tol).all()


def test_logits_graph_replays():
    """Captured and replayed on new inputs, with eager work between: every replay equals the eager call."""
    import torch
    import post_quantization_solver_amd as mpq
    z = torch.randn(9, 40000, device="cuda").bfloat16()
    tok = torch.randint(0, 40000, (9,), device="cuda").int()
    ids = torch.topk(z.float(), 20).indices.int()
    lp = torch.log_softmax(z.float(), 1).gather(1, ids.long())

    def both():
        a = mpq.token_logprobs(z, tok, top=20)
        b = mpq.distill(z, ids, lp, tail=True)
        return [a["logprob"], a["entropy"], a["top_ids"], a["top_logprobs"], b["loss"], b["grad"]]
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        z.copy_(torch.randn(9, 40000, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, both()):
            assert torch.equal(a, b), k


def test_logits_refusals():
    import torch
    import post_quantization_solver_amd as mpq
    z = torch.randn(4, 100, device="cuda")
    ids = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    lp = torch.zeros(4, 3, device="cuda")
    with pytest.raises(TypeError):
        mpq.token_logprobs(z.double())
    with pytest.raises(TypeError):
        mpq.token_logprobs(z.cpu())
    with pytest.raises(TypeError):
        mpq.token_logprobs(z, torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mpq.token_logprobs(z.t())
    with pytest.raises(ValueError):
        mpq.token_logprobs(z[:1].expand(4, 100))
    with pytest.raises(mpq.MPQError):
        mpq.token_logprobs(z, top=129)
    with pytest.raises(mpq.MPQError):
        mpq.distill(z, ids, lp, temperature=0.0)
    with pytest.raises(mpq.MPQError):
        mpq.distill(z, ids, lp, temperature=2.0, tail=True)
    with pytest.raises(ValueError):
        mpq.distill(z, ids, lp[:, :2].contiguous())
    with pytest.raises(TypeError):
        mpq.distill(z, ids, lp, grad=torch.empty(4, 100, device="cuda").half())
    with pytest.raises(mpq.MPQError):
        mpq.token_logprobs(z, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), top=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V,k,T,tail", [(5, 3, 1.0, True), (4099, 128, 2.0, False), (16391, 64, 1.0, True),
                                        (50257, 100, 4.0, False), (65537, 20, 1.0, True), (131072, 5, 1.0, True)])
def test_distill_many_rows(dtype, V, k, T, tail):
    """Enough rows for a workgroup each, around the widths that its registers hold."""
    g = np.random.default_rng(V)
    z = rows(g, 129, V, dtype, spread=2.5, pad=3, shift=1)
    ids, lp = teacher_list(g, z, k)
    check_distill(z, ids, lp, dtype, T, tail)


@pytest.mark.parametrize("V", [9001, 40003])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_many_rows_lists(V, tail):
    """Lists with gaps, repeats and zero masses, weights of 0, masked and extreme logits, in rows of a workgroup each."""
    import torch
    g = np.random.default_rng(V)
    z = rows(g, 140, V, "fp32", spread=2.0).clone()
    z[7, V - 5:] = float("-inf")
    z[8, ::2] = torch.finfo(torch.float32).min
    z[9] = z[9] * 1e6               # beyond what one fused step scales exactly
    z[10] = 0.5
    ids, lp = teacher_list(g, z, 70, noise=0.2)
    ids[0, 3:6] = [-1, V, 2 ** 31 - 1]
    ids[1, 5] = ids[1, 2]
    ids[1, 69] = ids[1, 2]
    lp[2, 4] = -np.inf
    ids[3] = -1
    ids[11, 1] = V - 1
    weights = (g.random(140) * 2).astype(np.float32).astype(np.float64)
    weights[4:6] = 0.0
    z[4] = float("nan")
    lp[9] = -4.0
    lp = np.maximum(lp, -60.0) + np.where(np.isinf(lp), -np.inf, 0.0).astype(np.float32)
    check_distill(z[:9].contiguous(), ids[:9], lp[:9], "fp32", 1.0, tail, weights[:9])
    keep = [i for i in range(140) if i != 9]
    check_distill(z[keep].contiguous(), ids[keep], lp[keep], "fp32", 1.0, tail, weights[keep])
    # row 9's masses: one token has all of the student's
    import post_quantization_solver_amd as mpq
    r = mpq.distill(z, dev(ids), dev(lp), tail=tail, weights=dev(weights.astype(np.float32)))
    _, grad, scale = R.distill(z[9:10].double().cpu().numpy(), ids[9:10], lp[9:10].astype(np.float64), 1.0, tail,
                               weights[9:10])
    assert np.isfinite(grad).all()
    assert (np.abs(host(r["grad"])[9] - grad[0]) <= 2.0 ** -16 * scale[0] + 1e-30).all()
