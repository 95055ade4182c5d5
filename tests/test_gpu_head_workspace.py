"""Calls stay within the workspace that their sizes ask for: what lies behind it is left alone."""
import numpy as np
import pytest

from test_gpu_head import inputs, packed_case
from test_gpu_linear import rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name,m,n,group", [("s16", 1003, 256, 0), ("s64", 700, 200, 0), ("e8240", 4099, 64, 0), ("e865536", 520, 520, 0),
                                            ("vec", 333, 264, 0), ("s16", 1003, 512, 128), ("s16", 300, 200, 33),
                                            ("matrix", 700, 128, 0), ("matrix", 517, 100, 0)])
@pytest.mark.parametrize("t", [1, 2, 4, 5, 70])
def test_within_its_size(dtype, name, m, n, group, t):
    import torch
    import post_quantization_solver_amd as mpq
    from post_quantization_solver_amd import binding as B
    lib, code = mpq.load_library(), dict(bf16=0, fp16=1, fp32=2)[dtype]
    g = np.random.default_rng(m + t)
    if name == "matrix":
        head = rows(g, m, n, dtype, scale=1.0 / np.sqrt(n))
        x, targets, b, w = inputs(g, m, n, t, dtype, True, False, 0, 0)
        size = lib.mpq_matrix_cross_entropy_workspace_bytes(code, t, m, n)
    else:
        head, x, targets, b, w, _ = packed_case(name, m, n, t, dtype, group=group, seed=t)
        size = lib.mpq_linear_cross_entropy_workspace_bytes(code, t, m, n, head.codebook.K, head.codebook.d, head.group)
    want = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w)
    ws = torch.full((size + (1 << 20),), 255, dtype=torch.uint8, device="cuda")
    for need_dx, need_dhead in ((True, True), (False, False), (True, False), (False, True)):
        got = mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, need_dx=need_dx, need_dhead=need_dhead,
                                       workspace=ws[:size])
        assert all(v is None or torch.equal(v, want[k]) for k, v in got.items())
        assert bool((ws[size:] == 255).all())
    if name[:2] != "e8":   # (the size knows a codebook's sizes, not its points: E8's decoder may need less than another's)
        with pytest.raises(B.MPQError):
            mpq.linear_cross_entropy(x, head, targets, bias=b, weights=w, workspace=ws[:size - 1])
