"""Host-side checks of the tuning step's C entries: sizes, and arguments refused
before anything reaches the GPU."""
import ctypes

import numpy as np

from oracle import ops_oracle as R
from post_quantization_solver_amd import binding as B
from test_abi import FAKE, lib  # noqa: F401

PLAN_MAGIC = 0x4d505141444d5731
NAN, INF = float("nan"), float("inf")


def tensors(*specs):
    full = [(1 << 20, 10, 0, 0.1, 0.0, 2, 0)] if not specs else specs
    return (B.AdamWTensor * len(full))(*(B.AdamWTensor(*s) for s in full)), len(full)


def spec(param=1 << 20, count=10, at=0, lr=0.1, wd=0.0, dtype=2, reserved=0):
    return param, count, at, lr, wd, dtype, reserved


def test_plan_sizes(lib):  # noqa: F811
    small = lib.mpq_adamw_plan_bytes(*tensors())
    assert small > 0 and small % 256 == 0
    assert lib.mpq_adamw_plan_bytes(*tensors(spec(count=10_000_000))) >= small + 4 * 4000
    assert lib.mpq_adamw_plan_bytes(None, 0) > 0
    for bad in ((spec(count=-1),), (spec(at=-256),), (spec(at=100),), (spec(count=(1 << 40) + 1),),
                (spec(count=257), spec(at=256)), (spec(at=512), spec(at=256)), (spec(at=(1 << 40) + 256),)):
        assert lib.mpq_adamw_plan_bytes(*tensors(*bad)) == 0
    assert lib.mpq_adamw_plan_bytes(None, 1) == 0 and lib.mpq_adamw_plan_bytes(tensors()[0], -1) == 0
    assert lib.mpq_adamw_plan_bytes(tensors()[0], (1 << 16) + 1) == 0


def test_plan_refusals(lib):  # noqa: F811
    def plan(*specs, table=FAKE, nb=1 << 30, out=True):
        P = B.AdamWPlan()
        return lib.mpq_adamw_plan(*tensors(*specs), table, nb, None, ctypes.byref(P) if out else None)
    assert plan(out=False) == -1 and plan(spec(param=None)) == -1
    assert plan(spec(count=-1)) == -2 and plan(spec(at=8)) == -2
    for bad in (dict(lr=-0.1), dict(lr=NAN), dict(lr=INF), dict(wd=-1.0), dict(wd=NAN), dict(dtype=3), dict(dtype=-1),
                dict(reserved=1), dict(param=(1 << 20) + 2)):
        assert plan(spec(**bad)) == -3, bad
    assert plan(spec(), spec(at=256)) == -3                                # the same memory twice
    assert plan(spec(), spec(param=(1 << 20) + 36, at=256)) == -3          # its last element
    assert plan(spec(), spec(param=(1 << 20) - 2, count=2, at=256, dtype=0)) == -3
    assert plan(nb=100) == -5 and plan(table=None) == -5 and plan(table=ctypes.c_void_p((1 << 20) + 8)) == -5


def test_step_refusals(lib):  # noqa: F811
    def step(plan=True, grads=True, magic=PLAN_MAGIC, beta1=0.9, beta2=0.99, eps=1e-8, scale=1.0, norm=0.0, lr=1.0, state=True,
             step=FAKE, m=FAKE, v=FAKE, ms=FAKE, vs=FAKE, elements=256, bits=8):
        P = B.AdamWPlan(1, 1, 256, 1 << 20, magic)
        S = B.AdamWState(step, m, v, ms, vs, elements, bits, 0)
        O = B.AdamWOptions(beta1, beta2, eps, scale, norm, lr, None, None)
        g = (ctypes.c_void_p * 1)(1 << 20) if grads else None
        return lib.mpq_adamw(ctypes.byref(P) if plan else None, g, ctypes.byref(O), ctypes.byref(S) if state else None, None)
    assert step(plan=False) == -1 and step(state=False) == -1 and step(grads=False) == -1 and step(step=None) == -1
    assert step(m=None) == -1 and step(v=None) == -1 and step(ms=None) == -1 and step(vs=None) == -1
    for bad in (dict(magic=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=NAN), dict(eps=0.0), dict(eps=NAN), dict(eps=1e-60),
                dict(eps=1e39), dict(scale=INF), dict(scale=NAN), dict(norm=-1.0), dict(norm=NAN), dict(lr=-1.0), dict(lr=INF),
                dict(bits=16)):
        assert step(**bad) == -3, bad
    assert step(elements=255) == -2
    assert step(m=ctypes.c_void_p((1 << 20) + 8)) == -5

    def moments(bits=8, elements=256, m=FAKE, out=FAKE, other=FAKE):
        S = B.AdamWState(FAKE, m, FAKE, FAKE, FAKE, elements, bits, 0)
        return lib.mpq_adamw_moments(ctypes.byref(S), out, other, None)
    assert lib.mpq_adamw_moments(None, FAKE, FAKE, None) == -1
    assert moments(bits=32) == -3 and moments(elements=100) == -2 and moments(m=None) == -1 and moments(out=None) == -1
    assert moments(other=ctypes.c_void_p((1 << 20) + 4)) == -5 and moments(elements=0) == 0


def test_struct_layout(tmp_path):
    """The binding's structs against the header's."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = ["#include <stddef.h>", '#include "mpq.h"']
    for cls, name in ((B.AdamWTensor, "mpq_adamw_tensor"), (B.AdamWPlan, "mpq_adamw_plan_t"), (B.AdamWState, "mpq_adamw_state"),
                      (B.AdamWOptions, "mpq_adamw_options")):
        lines.append(f'_Static_assert(sizeof({name}) == {ctypes.sizeof(cls)}, "{name}");')
        for f, _ in cls._fields_:
            lines.append(f'_Static_assert(offsetof({name}, {f}) == {getattr(cls, f).offset}, "{name}.{f}");')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\nint main(void) { return 0; }\n")
    r = subprocess.run([cc, "-std=c11", "-fsyntax-only", "-I", os.path.join(root, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_hash_is_even():
    """The rounding's random bits: even over their range, and unrelated between neighbours, halves and steps.

    2^20 words in 256 classes: 4096 each with a standard deviation of 64; correlations of 2^20 pairs have one of
    2^-10.  Five of them."""
    h = R.adamw_words(5, 3, 1 << 20, 1 << 20).astype(np.int64)
    for part in (h & 0xffff, h >> 16, R.mix(h ^ 0x9E3779B9).astype(np.int64) & 0xffff):
        assert np.abs(np.bincount(part >> 8, minlength=256) - 4096).max() < 5 * 64
    others = [np.roll(h, 1), R.adamw_words(5, 4, 1 << 20, 1 << 20).astype(np.int64),
              R.adamw_words(6, 3, 1 << 20, 1 << 20).astype(np.int64), R.adamw_words(5, 3, 1 << 32, 1 << 20).astype(np.int64)]
    for o in others:
        for a, b in ((h & 0xffff, o & 0xffff), (h >> 16, o >> 16)):
            assert abs(np.corrcoef(a, b)[0, 1]) < 5 * 2.0 ** -10
    assert abs(np.corrcoef(h & 0xffff, h >> 16)[0, 1]) < 5 * 2.0 ** -10


def test_codes_are_the_formats():
    """Oracle: every code decodes to itself, values between two codes go to either with the stated chance."""
    for F in (3, 4):
        L = R.code_levels(F)
        assert (np.diff(L) > 0).all() and L[-1] == (2 ** (F + 1) - 1) * 2.0 ** 14
        v = np.resize(L, -(-len(L) // 256) * 256).astype(np.float64)
        v[0] = L[-1]
        code, scale = R.encode8(v, F, np.full(len(v), 65535))
        assert scale[0] == 1.0 and np.array_equal(R.decode8(code, scale, F), v)


def head(lib, dtype=0, t=4, ldx=32, packed=FAKE, m=16, n=32, cb=None, scale=FAKE, group=0, targets=FAKE, loss=FAKE, x=FAKE,
         dx=FAKE, lddx=32, ds=FAKE, do=FAKE, db=FAKE, ws=FAKE, nb=1 << 40):
    from test_abi_ops import book
    cb = book() if cb is None else cb
    return lib.mpq_linear_cross_entropy(x, dtype, t, ldx, packed, m, n, ctypes.byref(cb), scale, None, group, None, targets,
                                        None, loss, dx, lddx, ds, do, db, ws, nb, None)


def matrix(lib, dtype=0, t=4, ldx=32, W=FAKE, ldw=32, m=16, n=32, targets=FAKE, loss=FAKE, x=FAKE, dx=FAKE, lddx=32, dW=FAKE,
           lddw=32, db=FAKE, ws=FAKE, nb=1 << 40):
    return lib.mpq_matrix_cross_entropy(x, dtype, t, ldx, W, ldw, m, n, None, targets, None, loss, dx, lddx, dW, lddw, db, ws,
                                        nb, None)


def test_head_refusals(lib):  # noqa: F811
    from test_abi_ops import book
    off = ctypes.c_void_p((1 << 20) + 8)
    for call in (head, matrix):
        assert call(lib, dtype=3) == -3 and call(lib, t=-1) == -2 and call(lib, t=1 << 22) == -2 and call(lib, m=0) == -2
        assert call(lib, n=0) == -2 and call(lib, ldx=31) == -2 and call(lib, lddx=31) == -2
        assert call(lib, x=None) == -1 and call(lib, targets=None) == -1 and call(lib, loss=None) == -1
        assert call(lib, db=None) == -1 and call(lib, ws=None) == -5 and call(lib, ws=off) == -5 and call(lib, nb=64) == -5
    assert head(lib, packed=None) == -1 and head(lib, packed=off) == -5 and head(lib, scale=None) == -1
    assert head(lib, do=None) == -1 and head(lib, ds=None) == -1
    assert head(lib, group=-1) == -3 and head(lib, group=8, cb=book(K=256, d=8)) == -4
    assert head(lib, cb=book(narrow=0)) == -4 and head(lib, cb=book(magic=1)) == -3
    assert matrix(lib, W=None) == -1 and matrix(lib, dW=None) == -1 and matrix(lib, ldw=31) == -2
    assert matrix(lib, lddw=31) == -2 and matrix(lib, m=(1 << 24) + 1) == -2 and matrix(lib, n=65537, ldx=1 << 17) == -2
    assert head(lib, t=0, dx=None, ds=None, do=None, db=None) == 0 and matrix(lib, t=0, dx=None, dW=None, db=None) == 0


def test_head_sizes(lib):  # noqa: F811
    f, g = lib.mpq_linear_cross_entropy_workspace_bytes, lib.mpq_matrix_cross_entropy_workspace_bytes
    for dtype in (0, 1, 2):
        for t in (0, 1, 17, 2048):
            assert f(dtype, t, 1000, 256, 16, 1, 0) > 0 and f(dtype, t, 1000, 256, 16, 1, 64) > 0
            assert f(dtype, t, 1000, 256, 65536, 8, 0) > 0 and g(dtype, t, 1000, 256) > 0
    assert f(3, 1, 10, 64, 16, 1, 0) == 0 and g(3, 1, 10, 64) == 0 and g(0, -1, 10, 64) == 0 and g(0, 1, 0, 64) == 0
    assert f(0, 1 << 22, 10, 64, 16, 1, 0) == 0 and f(0, 1, 10, 64, 16, 3, 0) == 0 and g(0, (1 << 22) - 1, 10, 65536) == 0
    # far from what the logits would take
    assert f(0, 1 << 16, 1 << 20, 4096, 65536, 8, 0) < 4 << 30
