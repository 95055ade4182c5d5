"""The few-token product waits for its table's loads by a count of the loads that
went out behind them (csrc/qskinny.hip).  A load that the compiler left out or
joined with another would make that count too large and the wait too short, so the
compiled kernels are read: behind the table's last load at least as many loads
stand as the wait before the first barrier leaves on their way."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")


def test_table_waits(tmp_path):
    from post_quantization_solver_amd import build as B
    out = str(tmp_path / "qskinny.s")
    r = subprocess.run([B.hipcc(), *[f for f in B.FLAGS if f != "-fPIC"], "-I", os.path.join(ROOT, "include"),
                        "--cuda-device-only", "-S", os.path.join(B.CSRC, "qskinny.hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    seen = 0
    for m in re.finditer(r"^(\S*q_skinny_kernelILi2E\S*):", text, re.M):
        lines = text[m.start():text.index(".Lfunc_end", m.start())].split("\n")
        barrier = next(k for k, line in enumerate(lines) if "s_barrier" in line)
        table = max(k for k, line in enumerate(lines[:barrier]) if "global_load_lds" in line)
        between = lines[table + 1:barrier]
        behind = sum(bool(re.search(r"\b(buffer|global)_load", line)) for line in between)
        left = [int(v) for v in re.findall(r"s_waitcnt vmcnt\((\d+)\)", "\n".join(between))]
        assert left and min(left) <= behind, (m.group(1), left, behind)
        seen += 1
    assert seen >= 8
