"""The tuning step's C entries at the ends of their arguments' ranges, before anything reaches the GPU."""
import ctypes

from post_quantization_solver_amd import binding as B
from test_abi import FAKE, lib  # noqa: F401
from test_abi_tune import PLAN_MAGIC


def test_eps_below_the_normal_range(lib):  # noqa: F811
    """Its reciprocal is infinite in float32, and an element without moments would become NaN."""
    def step(eps):
        plan = B.AdamWPlan(0, 0, 0, 1 << 20, PLAN_MAGIC)
        state = B.AdamWState(None, None, None, None, None, 0, 32, 0)   # (refused for `step` alone, after eps)
        options = B.AdamWOptions(0.9, 0.99, eps, 1.0, 0.0, 1.0, None, None)
        return lib.mpq_adamw(ctypes.byref(plan), None, ctypes.byref(options), ctypes.byref(state), None)
    for eps in (1e-39, 2.0 ** -127, 1e-44, 2.0 ** -149):
        assert step(eps) == -3, eps
    for eps in (2.0 ** -126, 1e-37, 1e-8, 1.0):
        assert step(eps) == -1, eps


def test_few_tokens_need_little(lib):  # noqa: F811
    """Up to four tokens of a packed head come straight from its codes: no operand planes, which were 252 to 541 MB here.

    A row of logits, the dx of some splits, and of column groups dz^T's operand (256 bytes a row of the head) and the
    contraction's parts (8 bytes for 64 weights): 64 MB at most for four tokens, 1 MB a token and some for rows."""
    f = lib.mpq_linear_cross_entropy_workspace_bytes
    for dtype in (0, 1, 2):
        for t in (1, 2, 4):
            for m in (32000, 128256):
                assert 4 * m * t < f(dtype, t, m, 4096, 65536, 8, 0) < (t + 8) << 20
                assert 4 * m * t < f(dtype, t, m, 4096, 16, 1, 0) < (t + 8) << 20
                assert 4 * m * t < f(dtype, t, m, 4096, 16, 1, 128) < 64 << 20
