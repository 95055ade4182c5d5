"""mpq_codebook keeps its layout: a caller that was built against an older header
hands mpq_codebook_prepare a struct of that size."""
import ctypes
import os
import shutil
import subprocess

import pytest

import post_quantization_solver_amd as mpq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = (("K", 0), ("d", 8), ("kind", 16), ("e8_qlast", 20), ("e8_last2", 24), ("tables", 56), ("magic", 64))


def test_binding_layout():
    C = mpq.binding.Codebook
    assert ctypes.sizeof(C) == 72
    assert tuple((name, getattr(C, name).offset) for name, _ in C._fields_) == FIELDS


def test_header_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include "mpq.h"\n' + "".join(
        f"_Static_assert(offsetof(mpq_codebook, {name}) == {at}, \"{name}\");\n" for name, at in FIELDS) +
        '_Static_assert(sizeof(mpq_codebook) == 72, "size");\nint main(void) { return 0; }\n')
    r = subprocess.run([cc, "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["s16", "e8240"])
def test_prepare_writes_the_struct_alone(name):
    """72 bytes of a longer buffer, and what is noted there tells packable codebooks apart."""
    import numpy as np
    import torch
    from test_gpu_linear import book
    lib = mpq.load_library()
    E = np.ascontiguousarray(book(name))
    K, d = E.shape
    tables = torch.empty(lib.mpq_codebook_bytes(K, d), dtype=torch.uint8, device="cuda")
    buf = (ctypes.c_ubyte * 96)(*([0xa5] * 96))
    cb = ctypes.cast(buf, ctypes.POINTER(mpq.binding.Codebook))
    rc = lib.mpq_codebook_prepare(E.ctypes.data_as(ctypes.c_void_p), K, d, tables.data_ptr(), tables.numel(),
                                  torch.cuda.current_stream().cuda_stream, cb)
    assert rc == 0 and bytes(buf[72:]) == b"\xa5" * 24
    assert cb.contents.narrow == (2 if d == 1 else 1) and mpq.prepare_codebook(E).struct.narrow == cb.contents.narrow
    if d == 1:
        assert mpq.prepare_codebook(E ** 2 / 255).struct.narrow == 0 and mpq.prepare_codebook(E ** 2).struct.narrow == 1
