"""Waits for the feed-forward kernels' transposing LDS reads, checked in this
repository's own gfx950 assembly (no GPU), as test_rr_asm_waits.py does for
the GEMM's: no instruction touches a register that such a read has not yet
delivered, on any path; a copy without the explicit waits must fail."""
import os
import re
import subprocess
import tempfile

import pytest

from tests.conftest import ROOT
from tests.test_rr_asm_waits import HIPCC, INC, check

SRC = os.path.join(ROOT, "tests", "host", "linear_asm_instances.hip")


def functions(asm):
    """{kernel symbol: [(kind, text)]} with kind 'label' or 'inst'."""
    funcs, cur = {}, None
    for raw in asm.splitlines():
        line = raw.split(";")[0].rstrip()
        m = re.match(r"^(_ZN2pg\w*linear_tile\w+):", line)
        if m:
            cur = funcs.setdefault(m.group(1), [])
            continue
        s = line.strip()
        if cur is None or not s:
            continue
        if s.startswith(".Lfunc_end"):
            cur = None
        elif re.match(r"^\.?L?\w+:$", s):
            cur.append(("label", s[:-1]))
        elif not s.startswith("."):
            cur.append(("inst", s))
    return funcs


@pytest.fixture(scope="module")
def kernels():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "linear.s")
        cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
               "-packed-fp32-ops", "--cuda-device-only", "-S", SRC, "-o", out] + ["-I" + p for p in INC]
        subprocess.run(cmd, check=True, capture_output=True)
        return functions(open(out).read())


def test_every_transposing_read_is_waited_for(kernels):
    assert len(kernels) == 20, sorted(kernels)
    for name, insts in kernels.items():
        assert any(k == "inst" and t.startswith("ds_read_b64_tr") for k, t in insts), name
        bad = check(insts)
        assert not bad, "%s: %s" % (name, bad[:3])


def test_deleted_waits_are_caught(kernels):
    for name, insts in kernels.items():
        without = [(k, t) for k, t in insts if not (k == "inst" and re.match(r"s_waitcnt .*lgkmcnt", t))]
        assert check(without), name
