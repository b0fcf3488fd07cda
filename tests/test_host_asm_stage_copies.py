"""In the large-tile kernels that stage E8M0 scales for several k-tiles at
once, every barrier that lets a k-tile be read waits for A's copy and for the
scale stage that the k-tile begins, on every path through the compiled code.
The sources are compiled to gfx950 assembly here (no GPU) and scanned; the
scanner is checked on planted cases first."""
import os
import tempfile

import pytest

import asm_stage_copies
from dense_gemm_packer_amd import build
from test_host_asm_copies import COPY, LOAD, ints

SCALES = "\tbuffer_load_dwordx4 v1, s[16:19], s8 offen lds\n"
WAIT3 = "\ts_waitcnt vmcnt(3)\n\ts_barrier\n"


def found(body, newer=1, ahead=1):
    return asm_stage_copies.find("k:\n" + body + "\ts_endpgm\n", lambda f: (newer, ahead))[0]


def test_scanner_finds_planted_waits():
    # A's copies as without scales; scale copies are loads like others
    assert not found(COPY + LOAD + COPY + LOAD + WAIT3)
    assert found(COPY + COPY + LOAD + WAIT3)
    assert not found(SCALES + COPY + LOAD + COPY + LOAD + WAIT3)
    # a stage in front of the first barrier is read behind it
    assert found(COPY + LOAD + COPY + SCALES + WAIT3 + COPY + LOAD + WAIT3)
    # one copied behind a barrier is read `ahead` barriers later: the barrier in
    # between does not wait for it, the next one does, or does not
    loop = COPY + LOAD + COPY + LOAD + WAIT3
    assert not found(loop + COPY + LOAD + SCALES + WAIT3 + COPY + COPY + LOAD + COPY + LOAD + WAIT3, newer=3)
    late = "\ts_waitcnt vmcnt(9)\n\ts_barrier\n"
    first = "\ts_waitcnt vmcnt(2)\n\ts_barrier\n"   # (covers what is in front of it)
    assert found(COPY + LOAD + COPY + LOAD + first + SCALES + LOAD + late + LOAD + COPY + LOAD + late, newer=9)
    assert not found(COPY + LOAD + COPY + LOAD + first + SCALES + LOAD + late + LOAD + COPY + LOAD + late, newer=9, ahead=2)
    # on one path of two
    branch = "\ts_cbranch_scc1 .LBB0_1\n" + 3 * LOAD + ".LBB0_1:\n"
    assert found(2 * COPY + 9 * LOAD + first + SCALES + 2 * LOAD + late + 5 * LOAD + branch + late, newer=9)
    assert not found(2 * COPY + 9 * LOAD + first + SCALES + 4 * LOAD + late + 5 * LOAD + branch + late, newer=9)


def w4(name):
    t = ints(name, "gemm_w4_kernel")      # <DT, SCALE, OUT, DB, SWZ, RA, ILV, SYNC, WM, TM, GR, XG>
    # a stage is read from behind the barrier in the k-tile before it on
    return (t[9] // 32, t[11] - 2) if t and t[11] else None


def tiled(name):
    t = ints(name, "gemm_tiled_kernel")   # <DT, TM, TN, WM, WN, KT, DEPTH, SCALE, OUT, PV, PD, GR, XG>
    return ((t[6] - 1) * (t[1] * t[5] // 1024) // (t[3] * t[4]), t[12] - 1) if t and t[12] else None


@pytest.mark.parametrize("src,plan,kernels", [("gemm_w4.hip", w4, 6), ("gemm_tiled.hip", tiled, 4)])
def test_barriers_cover_a_and_the_scale_stages(src, plan, kernels):
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        build.asm(src, out)
        text = open(out).read()
    bad, checked, scales = asm_stage_copies.find(text, plan)
    assert checked >= 2 * kernels and scales >= 2 * kernels
    assert not bad, (len(bad), bad[:5])
