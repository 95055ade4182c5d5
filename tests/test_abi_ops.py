"""Host-side checks of the operators' C entries: sizes, and arguments refused
before anything reaches the GPU."""
import ctypes

import pytest

import post_quantization_solver_amd as mpq
from test_abi import FAKE, fake_codebook, lib  # noqa: F401

BIG = 1 << 40
OFF = ctypes.c_void_p((1 << 20) + 8)


def book(narrow=1, **kw):
    cb = fake_codebook(**kw)
    cb.narrow = narrow
    return cb


def linear(lib, dtype=0, t=4, ldx=32, packed=FAKE, m=16, n=32, cb=None, scale=FAKE, offset=None, group=0, act=0, x=FAKE,
           res=None, ldr=16, y=FAKE, ldy=16, pre=None, ldp=16, ws=FAKE, nb=BIG):
    cb = book() if cb is None else cb
    return lib.mpq_linear(x, dtype, t, ldx, packed, m, n, ctypes.byref(cb), scale, offset, group, None, act, res, ldr, y,
                          ldy, pre, ldp, ws, nb, None)


def backward(lib, dtype=0, t=4, ldx=32, lddy=16, packed=FAKE, m=16, n=32, cb=None, scale=FAKE, group=0, act=0, dy=FAKE,
             x=FAKE, pre=None, ldp=16, dx=FAKE, lddx=32, ds=FAKE, do=FAKE, db=FAKE, ws=FAKE, nb=BIG):
    cb = book() if cb is None else cb
    return lib.mpq_linear_backward(dy, lddy, x, dtype, t, ldx, packed, m, n, ctypes.byref(cb), scale, None, group, act,
                                   pre, ldp, dx, lddx, ds, do, db, ws, nb, None)


def test_sizes(lib):  # noqa: F811
    assert lib.mpq_pack_bytes(16, 256, 65536, 8) == 1024
    assert lib.mpq_pack_bytes(17, 257, 16, 1) == 2 * 3 * 1024
    assert lib.mpq_pack_bytes(16, 64, 64, 1) == 1024
    assert lib.mpq_pack_bytes(0, 64, 64, 1) > 0
    for bad in ((-1, 64, 64, 1), (1, 0, 64, 1), (1, 65537, 64, 1), (1, 64, 65, 1), (1, 64, 1, 1), (1, 12, 8, 8),
                (1, 16, 65537, 8), (1, 16, 8, 3), ((1 << 24) + 1, 16, 8, 1)):
        assert lib.mpq_pack_bytes(*bad) == 0
    for fn in (lib.mpq_linear_workspace_bytes, lib.mpq_linear_backward_workspace_bytes):
        for t in (0, 1, 16, 1000):
            for m in (0, 1, 4096):
                assert fn(0, t, m, 64, 16, 1, 0) > 0
                assert fn(2, t, m, 64, 16, 1, 16) > 0
                assert fn(1, t, m, 64, 65536, 8, 0) > 0
        assert fn(3, 1, 1, 64, 16, 1, 0) == 0 and fn(0, 1 << 22, 1, 64, 16, 1, 0) == 0
        assert fn(0, -1, 1, 64, 16, 1, 0) == 0 and fn(0, 1, 1, 64, 16, 1, -1) == 0
        assert fn(0, 1, 1, 64, 65536, 8, 16) == 0
    for fn in (lib.mpq_token_logprobs_workspace_bytes, lib.mpq_distill_workspace_bytes):
        assert fn(0, 0, 1000, 4) > 0 and fn(2, 3, 1 << 20, 128) > 0
        assert fn(0, 1, 0, 4) == 0 and fn(0, 1, (1 << 20) + 1, 4) == 0 and fn(0, 1, 10, 129) == 0
        assert fn(0, 1, 10, -1) == 0 and fn(3, 1, 10, 1) == 0 and fn(0, -1, 10, 1) == 0
        assert fn(0, 1 << 31, 10, 1) == 0


def test_pack_refusals(lib):  # noqa: F811
    def pack(m=16, n=32, cb=None, codes=FAKE, packed=FAKE, nb=BIG):
        return lib.mpq_pack(codes, m, n, ctypes.byref(book() if cb is None else cb), packed, nb, None)
    assert pack(m=-1) == -2 and pack(n=0) == -2 and pack(m=0) == 0
    assert pack(codes=None) == -1 and pack(cb=book(tables=None)) == -1
    assert pack(cb=book(magic=0)) == -3 and pack(cb=book(narrow=0)) == -4
    assert pack(nb=8) == -5 and pack(packed=OFF) == -5 and pack(packed=None) == -5
    assert pack(n=30, cb=book(K=256, d=8)) == -2
    assert lib.mpq_pack(FAKE, 16, 32, None, FAKE, BIG, None) == -1


def test_linear_refusals(lib):  # noqa: F811
    assert linear(lib, dtype=3) == -3 and linear(lib, act=5) == -3 and linear(lib, act=-1) == -3
    assert linear(lib, group=-1) == -3 and linear(lib, group=8, cb=book(K=256, d=8)) == -4
    assert linear(lib, t=-1) == -2 and linear(lib, t=1 << 22) == -2 and linear(lib, ldx=31) == -2
    assert linear(lib, ldy=15) == -2 and linear(lib, res=FAKE, ldr=15) == -2 and linear(lib, pre=FAKE, ldp=15) == -2
    assert linear(lib, x=None) == -1 and linear(lib, y=None) == -1 and linear(lib, scale=None) == -1
    assert linear(lib, packed=None) == -1 and linear(lib, packed=OFF) == -5
    assert linear(lib, cb=book(narrow=0)) == -4 and linear(lib, cb=book(magic=1)) == -3
    assert linear(lib, ws=None) == -5 and linear(lib, nb=64) == -5 and linear(lib, ws=OFF) == -5
    assert linear(lib, t=0) == 0 and linear(lib, m=0, ldy=0) == 0


def test_backward_refusals(lib):  # noqa: F811
    assert backward(lib, dtype=-1) == -3 and backward(lib, act=9) == -3
    assert backward(lib, t=-1) == -2 and backward(lib, lddy=15) == -2 and backward(lib, lddx=31) == -2
    assert backward(lib, act=1, pre=FAKE, ldp=3) == -2
    assert backward(lib, act=1) == -1 and backward(lib, dy=None) == -1 and backward(lib, x=None) == -1
    assert backward(lib, do=None) == -1 and backward(lib, db=None) == -1
    assert backward(lib, ws=None) == -5 and backward(lib, nb=64) == -5
    assert backward(lib, t=0, dx=None, ds=None, do=None, db=None) == 0


def test_logit_refusals(lib):  # noqa: F811
    def lp(z=FAKE, dtype=0, t=2, V=10, ld=10, tok=FAKE, top=3, ws=FAKE, nb=BIG):
        return lib.mpq_token_logprobs(z, dtype, t, V, ld, tok, top, FAKE, None, None, None, None, ws, nb, None)
    assert lp(dtype=7) == -3 and lp(t=-1) == -2 and lp(V=0) == -2 and lp(ld=9) == -2 and lp(top=129) == -2
    assert lp(z=None) == -1 and lp(tok=None) == -1 and lp(nb=8) == -5 and lp(ws=OFF) == -5 and lp(t=0) == 0

    def ds(z=FAKE, t=2, V=10, ld=10, ids=FAKE, te=FAKE, k=3, T=1.0, tail=0, loss=FAKE, grad=FAKE, ldg=10, nb=BIG):
        return lib.mpq_distill(z, 0, t, V, ld, ids, te, k, T, tail, None, loss, grad, ldg, FAKE, nb, None)
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-45, 1e39):
        assert ds(T=T) == -3
    assert ds(T=2.0, tail=1) == -3
    assert ds(k=-1) == -2 and ds(k=129) == -2 and ds(ldg=9) == -2 and ds(ld=9) == -2
    assert ds(z=None) == -1 and ds(ids=None) == -1 and ds(te=None) == -1 and ds(loss=None) == -1
    assert ds(nb=8) == -5 and ds(t=0) == 0


def test_activations_match_header():
    import os
    import re
    txt = open(os.path.join(os.path.dirname(__file__), "..", "include", "mpq.h")).read()
    want = {n.lower(): int(v) for n, v in re.findall(r"#define MPQ_ACT_(\w+)\s+(\d+)", txt)}
    got = {"none" if k is None else k: v for k, v in mpq.binding.ACTIVATIONS.items()}
    assert got == want
