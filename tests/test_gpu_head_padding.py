"""Tokens that are not read, beside a head that holds NaN and infinities: their loss and gradient are zero all the same."""
import numpy as np
import pytest

from test_gpu_head import inputs, packed_case
from test_gpu_linear import rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["rows", "e8", "groups", "short groups", "matrix", "shifted matrix"])
@pytest.mark.parametrize("t", [1, 3, 4, 40, 33000])
def test_a_head_with_nan(kind, dtype, t):
    import torch
    import post_quantization_solver_amd as mpq
    m, n = (300, 128) if t < 1000 else (1100, 64)
    if kind.endswith("matrix"):
        g = np.random.default_rng(t)
        head = rows(g, m, n, dtype, 0, 1 if kind[0] == "s" else 0, scale=1.0 / np.sqrt(n))
        x, targets, b, w = inputs(g, m, n, t, dtype, True, False, 0, 0)
        spoilt, clean = head, head.clone()
    else:
        name, group = dict(rows=("s16", 0), e8=("e8240", 0), groups=("s16", 32))[kind.split()[-1]]
        if kind == "short groups":
            group = 8
        g = np.random.default_rng(t)
        head, *_ = packed_case(name, m, n, 2, dtype, group=group, seed=t)
        x, targets, b, w = inputs(g, m, n, t, dtype, True, False, 0, 0)
        spoilt, clean = head.scale, head.scale.clone()
    none = torch.zeros(t, dtype=torch.bool, device="cuda")
    none[::2] = True
    targets[::4] = -1
    w[2::4] = 0.0
    before = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    spoilt[7] = float("nan")
    spoilt[m - 1] = float("inf")
    for need_dhead in (True, False):
        got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dhead=need_dhead)
        assert not got["loss"][none].any() and not got["dx"][none].any()
        if t > 1:
            assert torch.isnan(got["loss"][~none]).all()
    # nobody reads it: no gradient for the head either
    targets.fill_(-1)
    got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    assert not any(v.any() for v in got.values())
    spoilt.copy_(clean)
    targets[1::2] = 3
    targets[::4] = -1
    again = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    assert not again["dx"][none].any() and all(torch.isfinite(v).all() for v in list(again.values()) + list(before.values()))


def test_an_autograd_graph_does_not_end_unnoticed():
    """x with a graph: its gradient is handed on by dx, or refused where none is wanted."""
    import torch
    import post_quantization_solver_amd as mpq
    head, x, targets, b, w, got = packed_case("s16", 100, 64, 5, "fp32", seed=3)
    leaf = (x / 2).requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        mpq.linear_cross_entropy(leaf * 2, head, targets, bias=b, weights=w, need_dx=False)
    y = leaf * 2
    y.backward(mpq.linear_cross_entropy(y, head, targets, bias=b, weights=w)["dx"])
    assert torch.equal(leaf.grad, 2 * got["dx"])
    with torch.no_grad():
        alone = mpq.linear_cross_entropy(leaf * 2, head, targets, bias=b, weights=w, need_dx=False)
    assert torch.equal(alone["loss"], got["loss"]) and torch.equal(alone["dscale"], got["dscale"])
    alone = mpq.linear_cross_entropy((leaf * 2).detach(), head, targets, bias=b, weights=w, need_dx=False)
    assert torch.equal(alone["loss"], got["loss"]) and alone["dx"] is None
