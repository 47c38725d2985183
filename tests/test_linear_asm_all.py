"""The waits that test_linear_asm_waits.py checks in some instances of the
feed-forward kernels, in every one that the library holds (their own sources,
compiled to gfx950 assembly; no GPU): transposing LDS reads, and sums that matrix
instructions in inline assembly leave in AGPRs."""
import concurrent.futures
import os
import subprocess

import pytest

from software_pipelined_tiled_02_amd import build
from tests.test_linear_asm_waits import functions, sums_too_early
from tests.test_rr_asm_waits import check

# source: kernels in all, of them with transposing reads, of them of 256 x 256 tiles
SOURCES = {"linear_rc.hip": (36, 0, 4), "linear_rr.hip": (36, 36, 4), "linear_gated.hip": (16, 0, 2),
           "linear_backward.hip": (18, 18, 2), "linear_weight.hip": (28, 28, 4)}
WIDE = "ELi256ELi256ELi"


def transposes(insts):
    return any(k == "inst" and t.startswith("ds_read_b64_tr") for k, t in insts)


def faults(insts, name):
    """What is read too early, as found by the two checks."""
    found = check(insts) if transposes(insts) else []
    return found + (sums_too_early(insts) if WIDE in name else [])


def look(source, folder):
    """(kernels, with transposing reads, wide ones, {kernel: faults})"""
    out = os.path.join(folder, source + ".s")
    subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out],
                   check=True, capture_output=True)
    with open(out) as f:
        kernels = functions(f.read())
    bad = {n: b[:3] for n, i in kernels.items() if (b := faults(i, n))}
    wide = {n: i for n, i in kernels.items() if WIDE in n}
    # a copy without the waits behind the last product must fail
    blind = [n for n, i in wide.items() if not sums_too_early([(k, t) for k, t in i if t != "s_nop 7"])]
    return len(kernels), sum(map(transposes, kernels.values())), len(wide), bad, blind


@pytest.fixture(scope="module")
def looked(tmp_path_factory):
    folder = str(tmp_path_factory.mktemp("asm"))
    with concurrent.futures.ProcessPoolExecutor(len(SOURCES)) as pool:
        jobs = {s: pool.submit(look, s, folder) for s in SOURCES}
        return {s: j.result() for s, j in jobs.items()}


@pytest.mark.parametrize("source", SOURCES)
def test_every_instance_waits(source, looked):
    kernels, transposing, wide, bad, blind = looked[source]
    assert (kernels, transposing, wide) == SOURCES[source]
    assert not bad and not blind, (bad, blind)
