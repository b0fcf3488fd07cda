"""No instruction reads or overwrites the result of an MFMA issued from inline
assembly before the MFMA has finished: the compiler does not see it as one and
inserts no wait.  The source is compiled to gfx950 assembly here (no GPU) and
every path from every MFMA scanned; the scanner is checked on planted cases
first."""
import os
import tempfile

import asm_results
from dense_gemm_packer_amd import build

MFMA = "v_mfma_f32_16x16x128_f8f6f4 a[0:3], v[4:11], v[12:19], a[0:3]"


def test_scanner_finds_planted_reads():
    head = "k:\n\t" + MFMA + "\n"
    assert asm_results.find(head + "\tv_accvgpr_read_b32 v2, a3\n")
    assert asm_results.find(head + "\ts_nop 7\n\tv_accvgpr_write_b32 a0, 0\n")
    assert not asm_results.find(head + "\ts_nop 7\n\ts_nop 2\n\tv_accvgpr_read_b32 v2, a3\n")
    assert not asm_results.find(head + "\tv_accvgpr_read_b32 v2, a4\n")
    assert not asm_results.find(head + "\t" + MFMA + "\n\ts_nop 7\n\ts_nop 2\n\tv_accvgpr_read_b32 v2, a3\n")
    # along a branch, and not past it
    assert asm_results.find(head + "\ts_cbranch_scc1 .LBB0_1\n\ts_endpgm\n.LBB0_1:\n\tds_write_b32 v0, a1\n")
    assert not asm_results.find(head + "\ts_branch .LBB0_1\n\tv_accvgpr_read_b32 v2, a3\n.LBB0_1:\n\ts_endpgm\n")


def test_accumulators_are_read_after_the_last_products():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        build.asm("gemm_w4.hip", out)
        text = open(out).read()
    assert "v_mfma" in text
    found = asm_results.find(text)
    assert not found, found[:5]
