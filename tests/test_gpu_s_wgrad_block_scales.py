"""GPU tests of the precision of a weight's gradient: x of fp32 block scales is held to
2^-17 whatever the result's type, and a bf16 result is the fp32 one rounded."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from gradient_common import GRAD_MODES, kept_values
from operand_common import EPS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def real(mode, rows, x_rows, n, k, seed):
    """(dC, X, sX, x in 64 bits): rows of different size, scales of all 24 bits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(x_rows, k, generator=g, device=DEV) * torch.exp(torch.randn(x_rows, 1, generator=g, device=DEV))
    X, S = (x.bfloat16(), None) if mode == "none" else dgp.quantize(x, GRAD_MODES[mode])
    return (1e-3 * torch.randn(rows, n, generator=g, device=DEV)).bfloat16(), X, S, kept_values(X, S, mode).to(DEV)


def check(got, d, x):
    """A block-scaled x to 2^-17 and fp32's own half step; fp32 sums of two products a row: at
    most 2 m roundings of a term and a few at the end; bf16's half step."""
    want, size = d.double().t() @ x, d.double().abs().t() @ x.abs()
    bound = size * (EPS * (2 * d.shape[0] + 9) + 2.0 ** -17)
    if got.dtype == torch.bfloat16:
        bound = bound + (want.abs() + bound) * 2.0 ** -8
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(1, 16, 128), (3, 144, 256), (16, 272, 640), (64, 128, 384), (20, 4112, 4096)])
def test_block_scales(out, m, n, k):
    dC, X, S, x = real("block128", m, m, n, k, m + n)
    check(dgp.gemm_wgrad(dC, X, S, dgp.SCALE_BLOCK128, out_dtype=out), dC, x)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k", [(144, 256), (1040, 1152)])
def test_block_scales_of_experts(out, gather, n, k):
    counts, tail = [5, 0, 40, 1, 18], 3
    m = sum(counts) + tail
    dC, X, S, x = real("block128", m, m // 2 if gather else m, n, k, 7)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    rows = torch.randint(0, X.shape[0], (m,), generator=torch.Generator().manual_seed(8)).to(torch.int32).to(DEV) if gather else None
    got = dgp.gemm_wgrad(dC, X, S, dgp.SCALE_BLOCK128, offsets=off.to(DEV), rows=rows, out_dtype=out)
    xr = x[rows.long()] if gather else x
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        check(got[e], dC[a:b], xr[a:b])


@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("m,n,k", [(33, 144, 256), (3000, 128, 256), (300, 4096, 3968)])
def test_a_bf16_result_is_the_fp32_one_rounded(mode, m, n, k):
    """The same products and sums in the same order, in one part and in several."""
    dC, X, S, _ = real(mode, m, m, n, k, 9)
    code = GRAD_MODES[mode]
    assert torch.equal(dgp.gemm_wgrad(dC, X, S, code, out_dtype=torch.bfloat16), dgp.gemm_wgrad(dC, X, S, code).bfloat16())
    off = torch.tensor([1, m // 2, m // 2, m], dtype=torch.int32, device=DEV)
    assert torch.equal(dgp.gemm_wgrad(dC, X, S, code, offsets=off, out_dtype=torch.bfloat16),
                       dgp.gemm_wgrad(dC, X, S, code, offsets=off).bfloat16())
