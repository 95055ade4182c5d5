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
