"""The ablation grid's output-head figures (output error, perplexity, divergence)
and one tuning step, against float64 formulas.

The product's error is sums of float32 (n = 128: 2^-20 of the terms' sum, here
about 2^-18 of a logit's size); a log probability adds float32's rounding of a
logit of some tens (2^-24 x 32).  2e-5 holds for nll and error.  The divergence is
a sum of some 65 products p log(p / q), each off by up to p x 2e-5: 4e-5 in all.
An Adam step's first move is lr g / (|g| + 1e-8): its sign is the gradient's
wherever the gradient stands clear of its own error (1e-4 of the largest).
"""
import numpy as np
import pytest

import mpq_synth as S
from oracle import ops_oracle as R
from parity_helpers import layer_tensors

pytestmark = pytest.mark.gpu

CASES = {
    "scalar3": lambda: S.make_layer("hd_s", 160, 128, seed=71, d=1, bits=3, power=0.5),
    "scalar4_g64": lambda: S.make_layer("hd_g", 96, 128, seed=72, d=1, bits=4, power=0.5, group=64),
    "lattice_k1000": lambda: S.make_layer("hd_l", 70, 64, seed=73, d=8, K=1000, power=0.6, r=60),
}


def formulas(ref, W):
    """error, nll, divergence of the logits x W^T (float64)."""
    x, z0 = ref["x"].double().cpu().numpy(), ref["logits"].double().cpu().numpy()
    ids, lp = ref["ids"].cpu().numpy().astype(np.int64), ref["logprobs"].double().cpu().numpy()
    z = x @ W.T
    lq = z - np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) - z.max(1, keepdims=True)
    nll = -lq[np.arange(len(z)), ref["targets"].cpu().numpy()].mean()
    p, q = np.exp(lp), np.exp(np.take_along_axis(lq, ids, 1))
    rest_p, rest_q = 1 - p.sum(1), 1 - q.sum(1)
    kl = (p * (lp - np.log(q))).sum(1)
    ok = rest_p > 1e-6
    kl[ok] += rest_p[ok] * np.log(rest_p[ok] / rest_q[ok])
    return np.linalg.norm(z - z0) / np.linalg.norm(z0), nll, kl.mean()


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("tokens", [1, 140])
def test_head_stats(name, tokens):
    import post_quantization_solver_amd as mpq
    from post_quantization_solver_amd.ablation import head_reference, head_stats
    L = CASES[name]()
    T = layer_tensors(L)
    ref = head_reference(T["W"], T["s"], T["V"], tokens, seed=5)
    assert ref["x"].shape == (tokens, L.n) and ref["ids"].shape == (tokens, min(64, L.m))
    z = ref["x"].double() @ T["W"].double().T
    assert float((ref["logits"].double() - z).norm() / z.norm()) < 1e-4
    codes = mpq.quantize_layer(T["W"], T["s"], T["V"], L.E, T["a"], T["o"], T_vamp=0, n_cd=1,
                               group=L.group or None)["codes"]
    layer = mpq.pack_layer(codes, L.E, T["a"], T["o"], group=L.group or None)
    got = head_stats(ref, layer)
    W = R.layer_weights(codes.cpu().numpy(), L.E, L.a, L.o, L.group)
    err, nll, kl = formulas(ref, W)
    assert abs(got["head_error"] - err) < 2e-5 and abs(got["head_nll"] - nll) < 2e-5
    assert abs(got["head_kl"] - kl) < 4e-5
    assert got["head_ppl"] == np.exp(got["head_nll"])


@pytest.mark.parametrize("name", list(CASES))
def test_tuning_step(name):
    """One step goes against the formula's gradient, in scale and offset."""
    import torch
    import post_quantization_solver_amd as mpq
    from post_quantization_solver_amd.ablation import head_reference, tune_affine
    L = CASES[name]()
    T = layer_tensors(L)
    ref = head_reference(T["W"], T["s"], T["V"], 50, seed=6)
    codes = mpq.quantize_layer(T["W"], T["s"], T["V"], L.E, T["a"], T["o"], T_vamp=0, n_cd=1,
                               group=L.group or None)["codes"]
    a, o = T["a"].clone(), T["o"].clone()
    lr = 2e-4 * float(a.abs().mean())
    tune_affine(ref, mpq.pack_layer(codes, L.E, a, o, group=L.group or None), 1)
    # the gradient by autograd in float64
    e, col = R.layer_entries(codes.cpu().numpy(), L.E, L.group)
    e, col = torch.from_numpy(np.ascontiguousarray(e)).double(), torch.from_numpy(np.ascontiguousarray(col)).long()
    a0, o0 = (T[k].double().cpu().reshape(L.m, -1).requires_grad_() for k in ("a", "o"))
    z = ref["x"].double().cpu() @ (a0[:, col] * e + o0[:, col]).T
    lq = torch.log_softmax(z, 1)
    lp, ids = ref["logprobs"].double().cpu(), ref["ids"].long().cpu()
    rest = (1 - lp.exp().sum(1)).clamp_min(1e-30)
    hidden = torch.zeros_like(lq, dtype=torch.bool).scatter_(1, ids, True)
    tail = rest * (rest.log() - torch.logsumexp(lq.masked_fill(hidden, -np.inf), 1))
    ((lp.exp() * (lp - lq.gather(1, ids))).sum(1) + tail).mean().backward()
    for got, start, ref_grad in ((a, T["a"], a0.grad), (o, T["o"], o0.grad)):
        moved = (got - start).double().cpu().reshape(L.m, -1)
        g = ref_grad
        clear = g.abs() > 1e-3 * g.abs().max()
        assert clear.float().mean() > 0.5
        assert (torch.sign(moved[clear]) == -torch.sign(g[clear])).all()
        want = -lr * g / (g.abs() + 1e-8)
        big = g.abs() > 1e-4 * max(float(g.abs().max()), 1e-2)
        # a float32 parameter near its start: half a step of its value, and a tenth for g's own error against eps
        slack = 2.0 ** -23 * start.double().cpu().reshape(L.m, -1).abs() + 0.1 * lr
        assert ((moved - want).abs() <= slack)[big].all()


def test_grid_with_a_head_keeps_the_rest():
    """The cells carry the head's figures, and everything else stays as without."""
    from post_quantization_solver_amd.ablation import markdown, run_grid
    L = CASES["scalar3"]()
    T = layer_tensors(L)
    before = {k: T[k].clone() for k in ("a", "o")}
    run = lambda **kw: run_grid(T["W"], T["s"], T["V"], L.E, T["a"], T["o"], (2,), (0, 1), L.damping,  # noqa: E731
                                log=lambda m: None, **kw)
    plain, full = run(), run(head_tokens=33, tune_steps=2)
    assert [c["cell"] for c in plain] == [c["cell"] for c in full]
    extra = {"head_error", "head_nll", "head_ppl", "head_kl", "head_ppl_original", "head_kl_tuned",
             "head_kl_tuning"}
    for p, f in zip(plain, full):
        assert set(f) - set(p) == extra and all(np.isfinite(f[k]) for k in extra)
        assert {k: v for k, v in p.items() if k != "seconds"} == {k: f[k] for k in p if k != "seconds"}
    assert all((T[k] == before[k]).all() for k in before)
    assert "head" not in markdown(plain, "t")
    lines = markdown(full, "t").splitlines()
    assert {line.count("|") for line in lines[2:]} == {15}
