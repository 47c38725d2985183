"""Waits that the feed-forward kernels see to themselves, checked in this
repository's own gfx950 assembly (no GPU).

Transposing LDS reads, as test_rr_asm_waits.py does for the GEMM's: no
instruction touches a register that such a read has not yet delivered, on any
path; a copy without the explicit waits must fail.

Matrix instructions written as inline assembly (sums in AGPRs): between the last
of them and any other instruction that touches an AGPR lie the 24 cycles of
s_nop that the kernel puts there, on any path, and between one that writes
an AGPR and the next matrix instruction at least 5."""
import os
import re
import subprocess
import tempfile

import pytest

from tests.conftest import ROOT
from tests.test_rr_asm_waits import HIPCC, INC, blocks, check

SRC = os.path.join(ROOT, "tests", "host", "linear_asm_instances.hip")


def functions(asm):
    """{kernel symbol: [(kind, text)]} with kind 'label' or 'inst'."""
    funcs, cur = {}, None
    for raw in asm.splitlines():
        line = raw.split(";")[0].rstrip()
        m = re.match(r"^(_ZN2pg\w*linear_(?:tile|few)\w+):", line)
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
    assert len(kernels) == 41, sorted(kernels)
    for name, insts in kernels.items():
        assert any(k == "inst" and t.startswith("ds_read_b64_tr") for k, t in insts), name
        bad = check(insts)
        assert not bad, "%s: %s" % (name, bad[:3])


def test_deleted_waits_are_caught(kernels):
    for name, insts in kernels.items():
        without = [(k, t) for k, t in insts if not (k == "inst" and re.match(r"s_waitcnt .*lgkmcnt", t))]
        assert check(without), name


def sums_too_early(insts):
    """Instructions that touch an AGPR less than 24 cycles of s_nop behind a
    matrix instruction on AGPRs, or such a one less than 5 behind a write."""
    bl = blocks(insts)
    index = {nm: k for k, (nm, _, _) in enumerate(bl)}
    state_in, work, bad = {0: (99, 99)}, [0], set()          # cycles of s_nop since a product, since a write
    while work:
        k = work.pop()
        product, write = state_in[k]
        for i, text in enumerate(bl[k][1]):
            mnem, _, ops = text.partition(" ")
            agprs = re.search(r"\ba(\[\d+:\d+\]|\d+)", ops) is not None
            if mnem == "s_nop":
                product, write = min(99, product + int(ops) + 1), min(99, write + int(ops) + 1)
            elif mnem.startswith("v_mfma") and agprs:
                if write < 5:
                    bad.add((bl[k][0], i, text))
                product, write = 0, 99
            elif agprs:
                if product < 24:
                    bad.add((bl[k][0], i, text))
                if mnem.startswith("v_accvgpr_write"):
                    write = 0
        for s in bl[k][2]:
            j = index.get(s)
            if j is not None:
                new = (product, write) if j not in state_in else tuple(map(min, state_in[j], (product, write)))
                if state_in.get(j) != new:
                    state_in[j] = new
                    work.append(j)
    return sorted(bad)


def test_sums_are_read_when_they_are_there(kernels):
    wide = {n: i for n, i in kernels.items() if "ELi256ELi256ELi" in n}
    assert len(wide) == 5, sorted(wide)
    for name, insts in wide.items():
        bad = sums_too_early(insts)
        assert not bad, "%s: %s" % (name, bad[:3])
        without = [(k, t) for k, t in insts if t != "s_nop 7"]
        assert sums_too_early(without), name
