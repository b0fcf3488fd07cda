"""Host-side choice of the grouped product's kernel by where its E8M0 scales
start (only invalid calls are made, so no device is touched)."""
import ctypes

import pytest

import test_host_operands as ops
from test_host_operands import L, P, dgp  # noqa: F401 (fixtures)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("which", ["sA", "sB"])
@pytest.mark.parametrize("tile_m", [64, 128])
def test_wide_scale_copies_need_whole_dwords(L, dgp, tile_m, which, off):
    """The one-wave-per-SIMD mxfp8 tiles of 64 and 128 rows copy scales 16 bytes
    at a time, and only so: they take neither K that is no multiple of 512 nor
    scales that start inside a dword."""
    cfg = ctypes.byref(dgp.Config(tile_m=tile_m, tile_n=256, tile_k=128, schedule=4))
    assert ops.grouped(L, K=640, cfg=cfg) == ops.CONFIG
    assert ops.grouped(L, K=512, cfg=cfg, **{which: P + off}) == ops.CONFIG


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("which", ["sA", "sB"])
def test_mxfp4_scales_start_at_whole_dwords(L, which, off):
    assert ops.grouped(L, dtype=ops.FP4, mode=ops.MX32, **{which: P + off}) == ops.ALIGN
