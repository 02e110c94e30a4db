"""The 256 x 256 tile kernel keeps its sums in accumulation registers that only its
assembly text names (csrc/k_head_wide.hip).  The build refuses code in which the
compiler uses one of them itself, and the kernel's products say what they write, so
that it does not at other optimisation levels either."""

import pytest

from matrix_optimizer_02_amd import build

SOUND = """
\tv_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], 0
\tds_read_b128 v[4:7], v1 ; a[0:15] in a comment
\tv_mfma_f32_32x32x16_bf16 a[0:15], v[4:7], v[8:11], a[0:15]
\tv_accvgpr_read_b32 v3, a[15]
\tv_accvgpr_read_b32 v3, a0
\t.set _ZN5dmuon.num_agpr, 256
"""


def test_products_and_reads_pass():
    build.check_accumulators(SOUND, "x")


@pytest.mark.parametrize("line", [
    "v_accvgpr_write_b32 a0, v0",
    "v_accvgpr_write_b32 a[2], v0",
    "v_accvgpr_mov_b32 a1, a0",
    "global_load_dword a7, v[0:1], off",
    "ds_write_b128 v0, a[0:3]",
    "scratch_store_dword off, a3, off",
    "v_mfma_f32_32x32x16_bf16 a[16:31], v[4:7], v[8:11], a[0:15]",
    "v_mfma_f32_32x32x16_bf16 a[0:15], a[16:19], v[8:11], a[0:15]",
])
def test_any_other_use_is_refused(line):
    with pytest.raises(RuntimeError, match="accumulation registers"):
        build.check_accumulators(SOUND + "\t" + line + "\n", "x")


def test_code_without_products_is_refused():
    with pytest.raises(RuntimeError, match="no product"):
        build.check_accumulators("\ts_endpgm\n", "x")


def test_the_kernel_holds_at_another_optimisation_level(tmp_path):
    # (-O3 is what every build checks; with -O1 the compiler is short of registers, and kept lanes'
    # offsets in a0 and a2 as long as the products did not say that they write there)
    for src in build.ASM_ACCUMULATORS:
        build.compile_hip(src, str(tmp_path / (src + ".o")), ["-O1"])
