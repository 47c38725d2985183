"""The build's table of kernel resources holds every kernel that the compiler reports on."""
import json

from software_pipelined_tiled_02_amd import build

REMARKS = """
a.hip:1:1: remark: Function Name: %s [-Rpass-analysis=kernel-resource-usage]
a.hip:1:1: remark:     VGPRs: %d [-Rpass-analysis=kernel-resource-usage]
a.hip:1:1: remark:     ScratchSize [bytes/lane]: %d [-Rpass-analysis=kernel-resource-usage]
a.hip:1:1: remark:     VGPRs Spill: %d [-Rpass-analysis=kernel-resource-usage]
"""


def test_every_reported_kernel_is_in_the_table(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "RESOURCES", str(tmp_path / "r.json"))
    gemm = build.kernel_symbol(0, 1, 0, 2, 1)
    norm = "_ZN2pg12_GLOBAL__N_119rms_backward_kernelILi3ELi1024ELi2ELb0ELb0EEEvNS_15RmsBackwardArgsE"
    build.write_resources({"a.hip": REMARKS % (gemm, 180, 0, 0), "b.hip": REMARKS % (norm, 128, 40, 9)})
    with open(build.RESOURCES) as f:
        table = json.load(f)
    assert table == {gemm: {"vgprs": 180, "scratch_bytes": 0, "vgpr_spill": 0},
                     norm: {"vgprs": 128, "scratch_bytes": 40, "vgpr_spill": 9}}
