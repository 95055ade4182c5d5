"""The gradients of a head's rows that no token makes likely, row by row against the formulas in float64.

Rows that lie up to 70 nats below the likeliest, by their biases: an optimizer that divides each element by its own
size sees their relative errors.  Tolerances:
  - a logit: (n / 16 + 32) 2^-22 sum |x a e| for the float32 sums, 2^-20 of it more where operands are two float16
    terms, and 2^-21 |b| for two operations on the bias; the logarithm of the mass is off by their mean under the
    probabilities; dz by both, relative, and 2^-16 for its exponential (|z - max| below 100);
  - dz^T times its token's factor (x's operand carries the inverse) is in float16 terms (2^-11 of an element for a
    bfloat16 matrix, 2^-19 for two with x's) under a power of two per row of the head: elements below 2^-28 of the
    row's bound lose up to 2^-39 of it, and a token's factor is its largest |x| to within 2: 2^-38 of the row's
    largest dz max |x|, times |x| over that maximum; x's elements likewise 2^-38 of their token's largest;
  - float32 sums over the tokens (t / 16 + 32) 2^-22, one rounding of the result.
"""
import numpy as np
import pytest

from parity_helpers import dev
from test_gpu_head import inputs, reference
from test_gpu_linear import STEP, make_layer, rows

pytestmark = pytest.mark.gpu


def check_rows(got, ref, bias, dtype, n, exact_terms, head=None):
    import torch
    V, t = len(ref["W"]), len(ref["x"])
    ax, adz = ref["ax"], ref["dz"].abs()
    logit = ((n / 16 + 32) * 2.0 ** -22 + (0.0 if exact_terms else 2.0 ** -20)) * (ax @ ref["A"].t().contiguous())
    logit = logit + 2.0 ** -21 * bias.abs().double()
    rel = logit + (torch.softmax(ref["z"], 1) * logit).sum(1, keepdim=True) + 2.0 ** -16
    ddz = adz * rel
    tops = ax.amax(1).clamp_min(1e-300)
    adzT, dzT = adz.t().contiguous(), ref["dz"].t().contiguous()
    M = adzT @ ax
    terms = 2.0 ** -11 if dtype == "bf16" and head is None else 2.0 ** -19
    E = ddz.t().contiguous() @ ax + (terms + (t / 16 + 32) * 2.0 ** -22) * M
    E = E + 2.0 ** -38 * ((adz * tops[:, None]).amax(0)[:, None] * (ax / tops[:, None]).sum(0)[None] + adzT @ tops[:, None])

    def within(name, value, want, tol, share):
        err = (value.double() - want).abs()
        assert not torch.isnan(value).any(), name
        worst = (err / tol.clamp_min(1e-300)).amax(1)
        assert (err <= tol).all(), (name, int(worst.argmax()), float(worst.max()))
        # (what the tolerance lets pass is not all there is)
        assert ((want.abs() > 2 * tol).double().mean(1) > 0.3).double().mean() > share, name
    if head is None:
        step, tiny = STEP[dtype], 2.0 ** -25 if dtype == "fp16" else 1e-38
        want = dzT @ ref["x"]
        within("dweight", got["dweight"], want, E + step * (want.abs() + E) + tiny, 0.1 if dtype == "fp16" else 0.9)
        return
    e, col, G = head["e"], head["col"], head["a"].shape[1]
    for name, ent in (("dscale", e), ("doffset", torch.ones_like(e))):
        def over_groups(v):
            return torch.zeros(V, G, dtype=torch.float64, device="cuda").index_add_(1, col, v)
        want = over_groups((dzT @ ref["x"]) * ent)
        within(name, got[name].reshape(V, G), want, over_groups(E * ent.abs()) + 2.0 ** -23 * want.abs() + 1e-38, 0.9)


def problem(g, m, n, t, dtype):
    """Targets among the likelier rows (a target's row is as large as its token), weights of very different sizes."""
    import torch
    x, targets, _, w = inputs(g, m, n, t, dtype, False, t > 2, 0, 0)
    w.mul_(dev(np.exp(2.0 * g.standard_normal(t)).astype(np.float32)))
    b = -70.0 * torch.arange(m, device="cuda") / m
    return x, targets.clamp_max(m // 50), b, w


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,n,t,pad", [(1000, 128, 1, 0), (1000, 96, 70, 0), (1003, 64, 300, 1), (2600, 64, 33000, 0)])
def test_matrix(dtype, m, n, t, pad):
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(m + t)
    W = rows(g, m, n, dtype, pad, 0, scale=1.0 / np.sqrt(n))
    x, targets, b, w = problem(g, m, n, t, dtype)
    got = mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w)
    check_rows(got, reference(x, dict(W=W), targets, b, w), b, dtype, n, dtype != "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("name,m,n,group,t", [("s16", 1000, 256, 128, 2), ("s16", 1003, 256, 64, 90), ("s64", 700, 96, 32, 200),
                                              ("s16", 2600, 128, 64, 33000), ("s16", 2570, 96, 32, 33000)])
def test_groups(dtype, name, m, n, group, t):
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(m + t)
    codes, E, scale, off = make_layer(name, m, n, group, t)
    scale = (scale * (4.0 / len(E))).astype(np.float32)
    off = (-scale * (len(E) / 2) + scale * g.standard_normal(scale.shape)).astype(np.float32)
    layer = mpq.pack_layer(dev(codes), E, dev(scale), dev(off), group=group)
    x, targets, b, w = problem(g, m, n, t, dtype)
    got = mpq.linear_cross_entropy(x, layer, targets, bias=b, weights=w)
    e = torch.from_numpy(np.asarray(E, np.float64)[codes].reshape(m, n)).cuda()
    G = -(-n // group)
    head = dict(e=e, a=layer.scale.double().reshape(m, G), o=layer.offset.double().reshape(m, G), mid=float(E[len(E) // 2, 0]),
                col=torch.arange(n, device="cuda") // group)
    check_rows(got, reference(x, head, targets, b, w), b, dtype, n, False, head)


def test_tokens_of_very_different_sizes():
    """Weights from 1e6 down to 1e-12 beside x from 1e-6 up to 3: a row's bound is of their products."""
    import torch
    import post_quantization_solver_amd as mpq
    g = np.random.default_rng(2)
    m, n, t = 500, 64, 40
    W = rows(g, m, n, "fp32", scale=1.0 / np.sqrt(n))
    x, targets, b, w = problem(g, m, n, t, "fp32")
    x.mul_(torch.logspace(-6, 0.5, t, device="cuda")[:, None])
    w.mul_(torch.logspace(6, -12, t, device="cuda"))
    got = mpq.linear_cross_entropy(x, W, targets, bias=b, weights=w)
    check_rows(got, reference(x, dict(W=W), targets, b, w), b, "fp32", n, False)
