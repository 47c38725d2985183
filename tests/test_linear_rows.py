"""Host check of what tells operands that overlap from those that do not (no
GPU); see tests/host/check_linear_rows.cpp."""
import os
import subprocess
import tempfile

from tests.conftest import ROOT


def test_rows_meet_where_they_have_a_byte_in_common():
    src = os.path.join(ROOT, "tests", "host", "check_linear_rows.cpp")
    inc = os.path.join(ROOT, "software_pipelined_tiled_02_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", inc, src, "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True)
        assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout
