"""CPU check of the offsets by which the linear attention walk reads its
operands' rows (csrc/walk_rows.hpp): builds tests/walk_rows_check.cpp as a host
program against the library's own header and runs it."""
import os
import subprocess

import pytest

from tests.test_epoch import CSRC, ROOT, _hipcc


def test_rows_hold_only_their_own_elements(tmp_path):
    cc = _hipcc()
    if cc is None:
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "walk_rows_check")
    src = os.path.join(ROOT, "tests", "walk_rows_check.cpp")
    r = subprocess.run([cc, "-O2", "-std=c++17", "-I", CSRC, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
