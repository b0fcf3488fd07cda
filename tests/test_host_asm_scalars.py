"""Global -> LDS copies written in inline assembly read no scalar register that
a vector instruction wrote too shortly before, and the products written so keep
their own wait states: the weight gradient's source is compiled to gfx950
assembly here (no GPU) and scanned; the scanner is checked on planted cases first."""
import os
import tempfile

import asm_hazards
import asm_results
import asm_scalars
from dense_gemm_packer_amd import build

COPY = "\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"


def test_scanner_finds_planted_reads():
    head = "k:\n"
    assert asm_scalars.find(head + "\tv_readlane_b32 s5, v9, 3\n\ts_nop 3\n" + COPY)
    assert not asm_scalars.find(head + "\tv_readlane_b32 s5, v9, 3\n\ts_nop 4\n" + COPY)
    assert not asm_scalars.find(head + "\tv_readlane_b32 s8, v9, 3\n" + COPY)           # another register
    assert asm_scalars.find(head + "\tv_cmp_lt_i64_e64 s[6:7], v[2:3], v[4:5]\n" + COPY)
    assert asm_scalars.find(head + "\tv_add_co_u32_e64 v2, s[6:7], v2, v3\n" + COPY)
    assert not asm_scalars.find(head + "\ts_add_u32 s5, s5, s9\n" + COPY)               # a scalar write
    # across a loop's back edge
    assert asm_scalars.find(head + ".LBB0_1:\n" + COPY + "\tv_readlane_b32 s5, v9, 3\n\ts_cbranch_scc1 .LBB0_1\n")


def test_weight_gradient_keeps_the_wait_states():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        build.asm("wgrad.hip", out)
        text = open(out).read()
    assert "v_mfma" in text and "offen lds" in text
    for scan in (asm_scalars, asm_hazards, asm_results):
        found = scan.find(text)
        assert not found, found[:5]
