"""Host check of the form that the norm's backward pass takes (no GPU): at
every size and type one that takes that size; see tests/host/check_rms_plan.cpp."""
import os
import subprocess
import tempfile

from tests.conftest import ROOT


def test_backward_form_takes_the_size_it_is_given():
    src = os.path.join(ROOT, "tests", "host", "check_rms_plan.cpp")
    inc = os.path.join(ROOT, "software_pipelined_tiled_02_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "check")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", inc, src, "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True)
        assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout
