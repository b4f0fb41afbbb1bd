"""The build's check of the compiler's resource report (CPU): kernels that may not
use scratch memory."""
import pytest

from group_wise_affine_amd import build


def report(*kernels):
    """As hipcc prints it: one remark per line and figure."""
    tail = f" [{build.REPORT}]"
    out = []
    for name, scratch, spill in kernels:
        for what, v in (("Function Name", name), ("    TotalSGPRs", 90), ("    VGPRs", 256), ("    AGPRs", 17),
                        ("    ScratchSize [bytes/lane]", scratch), ("    Dynamic Stack", False),
                        ("    Occupancy [waves/SIMD]", 1), ("    SGPRs Spill", 33), ("    VGPRs Spill", spill),
                        ("    LDS Size [bytes/block]", 512)):
            out.append(f"/a/kv8_attn.hip:607:1: remark: {what}: {v}{tail}")
    return "warning: something else\n" + "\n".join(out) + "\n"


def test_kernels_without_scratch_pass():
    build.check_no_scratch("kv8_attn.hip", report(("a", 0, 0), ("b", 0, 0)))   # (scalar spills go to vector lanes)


@pytest.mark.parametrize("bad", [("b", 8, 1), ("b", 0, 1), ("b", 16, 0)])
def test_a_spilling_kernel_fails_the_build(bad):
    with pytest.raises(RuntimeError, match="b: "):
        build.check_no_scratch("kv8_attn.hip", report(("a", 0, 0), bad, ("c", 0, 0)))


@pytest.mark.parametrize("text", ["", "warning: nothing said of registers\n", report(("a", 0, 0)).replace("VGPRs Spill", "")])
def test_no_report_fails_the_build(text):
    with pytest.raises(RuntimeError, match="reported no"):
        build.check_no_scratch("kv8_attn.hip", text)


def test_the_attention_is_checked():
    assert "kv8_attn.hip" in build.NO_SCRATCH and build.NO_SCRATCH <= set(build.SOURCES)
