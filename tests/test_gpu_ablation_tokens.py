"""The ablation grid's tuning on tokens: cross entropy of the layer read as a head, and AdamW
steps, against float64 formulas.

A first AdamW step without decay moves a parameter by lr g / (|g| + eps), with 8-bit
moments too (they are rounded after it): its sign is the gradient's wherever the gradient
stands clear of its own error (1e-3 of the largest), and its size to a tenth where |g| is
a hundred times eps and more.
"""
import numpy as np
import pytest

from oracle import ops_oracle as R
from parity_helpers import layer_tensors
from test_gpu_ablation_head import CASES

pytestmark = pytest.mark.gpu


def gradient(ref, codes, L, a, o):
    """The mean loss over the drawn tokens and its gradients by autograd in float64."""
    import torch
    e, col = R.layer_entries(codes.cpu().numpy(), L.E, L.group)
    e, col = torch.from_numpy(np.ascontiguousarray(e)).double(), torch.from_numpy(np.ascontiguousarray(col)).long()
    a, o = (t.double().cpu().reshape(L.m, -1).clone().requires_grad_() for t in (a, o))
    z = ref["x"].double().cpu() @ (a[:, col] * e + o[:, col]).T
    loss = torch.nn.functional.cross_entropy(z, ref["targets"].long().cpu())
    loss.backward()
    return float(loss.detach()), a.grad, o.grad


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name", list(CASES))
def test_tuning_step_on_tokens(name, bits):
    import torch
    import post_quantization_solver_amd as mpq
    from post_quantization_solver_amd.ablation import head_reference, tune_affine_on_tokens
    L = CASES[name]()
    T = layer_tensors(L)
    ref = head_reference(T["W"], T["s"], T["V"], 50, seed=6)
    codes = mpq.quantize_layer(T["W"], T["s"], T["V"], L.E, T["a"], T["o"], T_vamp=0, n_cd=1,
                               group=L.group or None)["codes"]
    a, o = T["a"].clone(), T["o"].clone()
    lr = 2e-4 * float(a.abs().mean())
    layer = mpq.pack_layer(codes, L.E, a, o, group=L.group or None)
    loss0, ga, go = gradient(ref, codes, L, a, o)
    losses = tune_affine_on_tokens(ref, layer, 1, state_bits=bits)
    assert losses.shape == (1,) and abs(float(losses[0]) - loss0) <= 1e-5 * max(1.0, loss0)
    for got, start, g in ((a, T["a"], ga), (o, T["o"], go)):
        moved = (got - start).double().cpu().reshape(L.m, -1)
        clear = g.abs() > 1e-3 * g.abs().max()
        assert clear.float().mean() > 0.3
        assert (torch.sign(moved[clear]) == -torch.sign(g[clear])).all()
        want = -lr * g / (g.abs() + 1e-8)
        big = g.abs() > max(1e-4 * float(g.abs().max()), 1e-6)
        # a float32 parameter near its start: half a step of its value, and a tenth for g's own error
        slack = 2.0 ** -23 * start.double().cpu().reshape(L.m, -1).abs() + 0.1 * lr
        assert ((moved - want).abs() <= slack)[big].all()
    more = tune_affine_on_tokens(ref, layer, 3, state_bits=bits, max_norm=1.0)
    assert torch.isfinite(more).all() and torch.isfinite(a).all() and torch.isfinite(o).all()


def test_grid_tuned_on_tokens():
    """The cells carry the same figures as with the other tuning, and the affine stays the grid's."""
    from post_quantization_solver_amd.ablation import run_grid
    L = CASES["scalar3"]()
    T = layer_tensors(L)
    before = {k: T[k].clone() for k in ("a", "o")}
    cells = {on: run_grid(T["W"], T["s"], T["V"], L.E, T["a"], T["o"], (2,), (0, 1), L.damping, log=lambda m: None,
                          head_tokens=33, tune_steps=2, tune_on=on, state_bits=8) for on in ("divergence", "tokens")}
    for p, q in zip(cells["divergence"], cells["tokens"]):
        assert set(p) == set(q) and all(np.isfinite(q[k]) for k in ("head_kl_tuned", "head_kl_tuning"))
        assert {k: v for k, v in p.items() if k not in ("seconds", "head_kl_tuned", "head_kl_tuning")} == \
            {k: q[k] for k in p if k not in ("seconds", "head_kl_tuned", "head_kl_tuning")}
    assert all((T[k] == before[k]).all() for k in before)
