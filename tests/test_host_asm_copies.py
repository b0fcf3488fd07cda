"""Every barrier of the large-tile kernels that lets a k-tile of A be read
waits for its asynchronous copy, on every path through the compiled code.  The
sources are compiled to gfx950 assembly here (no GPU) and scanned; the scanner
is checked on planted cases first."""
import os
import re
import tempfile

import pytest

import asm_copies
from dense_gemm_packer_amd import build

COPY = "\tbuffer_load_dwordx4 v1, s[4:7], s8 offen lds\n"
LOAD = "\tbuffer_load_dwordx4 v[4:7], v2, s[12:15], 0 offen\n"


def found(body, newer=1):
    return asm_copies.find("k:\n" + body + "\ts_endpgm\n", lambda f: newer)[0]


def test_scanner_finds_planted_waits():
    wait = "\ts_waitcnt vmcnt(3)\n\ts_barrier\n"
    assert not found(COPY + LOAD + COPY + LOAD + wait)            # the first copy has three loads behind it
    assert found(COPY + COPY + LOAD + wait)                       # one was removed
    assert not found(COPY + COPY + LOAD + "\ts_waitcnt vmcnt(2) lgkmcnt(0)\n" + wait)
    assert not found("\ts_waitcnt vmcnt(0)\n" + COPY + wait)      # the copy that may be outstanding
    loop = COPY + LOAD + ".LBB0_1:\n" + COPY + LOAD + wait + "\ts_cbranch_scc1 .LBB0_1\n"
    assert not found(loop)
    assert found(COPY + LOAD + "\ts_cbranch_scc1 .LBB0_2\n" + LOAD + ".LBB0_2:\n" + COPY + wait)   # one path of two


def ints(name, kernel):
    m = re.match(r"_ZN3dgp\d+" + kernel + r"I((?:Li\d+E)+)E", name)
    return [int(v) for v in re.findall(r"Li(\d+)E", m.group(1))] if m else None


def w4(name):
    t = ints(name, "gemm_w4_kernel")      # <DT, SCALE, OUT, DB, SWZ, RA, ILV, SYNC, WM, TM, GR, XG>
    return t[9] // 32 if t and not t[7] and not t[11] else None


def tiled(name):
    t = ints(name, "gemm_tiled_kernel")   # <DT, TM, TN, WM, WN, KT, DEPTH, SCALE, OUT, PV, PD, GR, XG>
    return (t[6] - 1) * (t[1] * t[5] // 1024) // (t[3] * t[4]) if t and not t[12] else None


@pytest.mark.parametrize("src,newer", [("gemm_w4.hip", w4), ("gemm_tiled.hip", tiled)])
def test_barriers_cover_their_copies(src, newer):
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        build.asm(src, out)
        text = open(out).read()
    bad, checked = asm_copies.find(text, newer)
    assert checked > 50
    assert not bad, (len(bad), bad[:5])
