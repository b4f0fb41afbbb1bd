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


BLOCK = """\t;;#ASMSTART
\ts_nop 1
\tv_mfma_i32_32x32x32_i8 a[0:15], v[2:5], v[6:9], a[0:15]
\ts_waitcnt lgkmcnt(0)
%s\t;;#ASMEND
"""
PLAIN = BLOCK % ""
LAST = BLOCK % "\ts_cmp_lg_u32 s8, 0\n\ts_cbranch_scc1 .Lgo1\n\ts_nop 15\n\ts_nop 15\n.Lgo1:\n"
ADDRESS = "\tv_add_u32_e32 v44, 1, v45   ; a0 is not meant\n"
MOVE = "\tv_accvgpr_read_b32 v2, a0\n"
STORE = "\tglobal_store_dwordx4 v[0:1], a[0:3], off\n"


def kernel(before="\tv_accvgpr_write_b32 a0, 0\n", top=ADDRESS, between=ADDRESS, last=LAST, tail="\ts_add_i32 s8, s8, -1\n",
           after=MOVE):
    return ("_Z4kernv:   ; @_Z4kernv\n" + before + ".LBB0_1:\n" + top + PLAIN + between + last + tail +
            "\ts_cbranch_scc1 .LBB0_1\n" + after + "\ts_endpgm\n.Lfunc_end0:\n")


def test_products_in_assembly_pass():
    build.check_products("i8.hip", kernel())


@pytest.mark.parametrize("where", ["top", "between", "tail"])
@pytest.mark.parametrize("what", [MOVE, STORE])
def test_a_sum_touched_between_products_fails_the_build(where, what):
    with pytest.raises(RuntimeError, match="between products"):
        build.check_products("i8.hip", kernel(**{where: what}))


def test_products_without_a_wait_fail_the_build():
    with pytest.raises(RuntimeError, match="no wait"):
        build.check_products("i8.hip", kernel(last=PLAIN))
    with pytest.raises(RuntimeError, match="no matrix products"):
        build.check_products("i8.hip", kernel().replace("v_mfma", "v_add"))


def test_the_tile_product_is_checked():
    assert "i8.hip" in build.ASM_PRODUCTS and build.ASM_PRODUCTS <= set(build.SOURCES)
