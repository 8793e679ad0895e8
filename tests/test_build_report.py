"""The build's look at the compiler's report of a kernel's resources."""
import pytest

from lossless_float_weight_amd import build


def report(*kernels):
    lines = []
    for name, scratch, sgpr, vgpr in kernels:
        for what, n in (("Function Name", name), ("    VGPRs", 128), ("    ScratchSize [bytes/lane]", scratch),
                        ("    SGPRs Spill", sgpr), ("    VGPRs Spill", vgpr)):
            lines.append(f"a.hip:1:0: remark: {what}: {n} [-Rpass-analysis=kernel-resource-usage]")
    return "\n".join(lines)


def test_spills_are_found():
    clean = ("_Z10k_mx_tiledILi2E", 0, 0, 0)
    assert build.spilling(report(clean), "k_mx_tiled") == []
    assert build.spilling(report(("_Z5other", 64, 3, 16), clean), "k_mx_tiled") == []
    for bad in ((16, 0, 4), (0, 1, 0), (0, 0, 1), (8, 0, 0)):
        got = build.spilling(report(clean, ("_Z10k_mx_tiledILi3E", *bad), ("_Z5other", 0, 0, 0)), "k_mx_tiled")
        assert len(got) == sum(v != 0 for v in bad) and all("ILi3E" in g for g in got)


def test_a_report_without_the_kernel_is_an_error():
    with pytest.raises(RuntimeError):
        build.spilling(report(("_Z5other", 0, 0, 0)), "k_mx_tiled")
    with pytest.raises(RuntimeError):
        build.spilling("", "k_mx_tiled")
