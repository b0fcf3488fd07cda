"""GPU tests of the grouped product's E8M0 scales at addresses that a view into
a larger buffer may have, on every compiled tile."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from operand_common import MODES
from test_gpu_j_grouped import TILES, aligned_loss, check, config, operands

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def at_byte(t, off):
    """A copy of t that starts `off` bytes past a 16-byte boundary, between bytes
    that would make every product they scale a NaN."""
    buf = torch.full((t.numel() + 64,), 255, dtype=torch.uint8, device=DEV)
    view = buf[16 + off:16 + off + t.numel()]
    view.copy_(t.flatten())
    assert view.data_ptr() % 16 == off
    return view.view(t.shape)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("mode,tile,k,off_a,off_b", [
    (mode, tile, k, a, b)
    for mode, shifts in (("mx128", ((512, 1, 0), (512, 0, 3), (1536, 2, 1))), ("mx32", ((512, 4, 0), (768, 0, 12), (768, 8, 4))))
    for tile in (None, *TILES[mode]) for k, a, b in shifts])
def test_scales_at_any_byte(mode, tile, k, off_a, off_b, gather):
    """MX128 scales may start at any byte, MX32 scales at any dword: the bits of
    the same call on aligned scales, and the 64-bit product."""
    counts, n = [5, 0, 33, 1, 300, 0, 17], 384
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    m = offsets[-1]
    a_rows = m // 2 if gather else m
    A, sA, Bs, sB, ad, bd = operands(mode, a_rows, len(counts), n, k, 53)
    rows = torch.randint(0, a_rows, (m,), generator=torch.Generator().manual_seed(54)) if gather else None
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    idx = None if rows is None else rows.to(torch.int32).to(DEV)
    want = dgp.gemm_preshuffle_grouped(A, Bs, off, sA, sB, MODES[mode], rows=idx, config=config(tile))
    got = dgp.gemm_preshuffle_grouped(A, Bs, off, at_byte(sA, off_a), at_byte(sB, off_b), MODES[mode], rows=idx,
                                      config=config(tile))
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    check(got, got.cpu(), ad, bd, offsets, rows, k, aligned_loss if mode == "mx128" else None)
