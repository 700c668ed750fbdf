"""The build's look at the accumulation registers of the 4-bit products (CPU): their sums stand there by name, which
the compiler does not know."""
from __future__ import annotations

import os

import pytest

from rank_gradient_compression_powersgd_amd import build as b

GOOD = """
0000000000001000 <kernel>:
\tv_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[44:47], v[4:7], a[0:3], v166, v168 op_sel_hi:[0,0,0] cbsz:4 blgp:4// 0098B8: D3AC0000
\tv_mfma_f32_16x16x32_bf16 a[252:255], v[44:47], v[4:7], 0     // 0098C8: D3AC1000 a5
\tv_accvgpr_read_b32 v2, a0                                  // 00BBC4: D3D84002 18000100
\tglobal_store_dwordx4 v[2:3], v[4:7], off offset:16
\ts_add_u32 s0, s1, s2
"""


def test_products_and_reads_of_sums_pass():
    assert b.foreign_accumulation(GOOD) == []


@pytest.mark.parametrize("line", ["v_accvgpr_write_b32 a3, v0", "v_accvgpr_mov_b32 a1, a2", "global_load_dwordx4 a[4:7], v[0:1], off",
                                  "ds_read_b128 a[0:3], v1", "global_store_dwordx4 v[2:3], a[4:7], off", "scratch_load_dword a9, off, s32"])
def test_anything_else_is_found(line):
    assert b.foreign_accumulation(GOOD + "\t" + line + "   // 00BBC4: D3D84002\n") == [line]


def test_the_built_products():
    obj = os.path.join(b.BUILD, "k_mx_gemm.o")
    if not os.path.exists(obj):
        pytest.skip("the library was built elsewhere: no object file")
    text = b.disassembly(obj)
    # every tile's kernel is there, and what is looked for
    assert text.count("k_mx_gemm") >= 12 and text.count("v_mfma_scale_f32_16x16x128_f8f6f4") > 500 and "v_accvgpr_read_b32 v" in text
    b.check_named_sums(obj)
