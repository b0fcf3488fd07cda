"""GPU tests of the gradients' entry points for M = 0 as a caller of the C ABI may
make them: no inputs at all and strides that nothing is read with."""
import pytest
import torch

import dense_gemm_packer_amd as dgp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, BF16, F32 = dgp.FP8_E4M3, dgp.BF16, dgp.F32


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("ldc", [0, -64, 8, 128])
@pytest.mark.parametrize("mode,dtype", [(dgp.SCALE_NONE, BF16), (dgp.SCALE_TENSOR, E4M3), (dgp.SCALE_BLOCK128, E4M3), (dgp.SCALE_MX128, E4M3)])
@pytest.mark.parametrize("n,k,e", [(144, 256, 1), (16, 128, 3), (1040, 1152, 2)])
def test_wgrad(ldc, mode, dtype, n, k, e):
    off = torch.zeros(e + 1, dtype=torch.int32, device=DEV) if e > 1 else None
    out = torch.full((e, n, k), 7.0, device=DEV)
    for accumulate in (1, 0):
        status = dgp.lib().dgp_gemm_wgrad(None, ldc, None, 0, dtype, None, mode, out.data_ptr(), F32, accumulate, 0, n, k, e,
                                          None if off is None else off.data_ptr(), None, None, 0, stream())
        assert status == 0
        assert bool((out == (7.0 if accumulate else 0.0)).all())


@pytest.mark.parametrize("k", [256, 9216])
def test_norms(k):
    dw, db = torch.full((2, k), 7.0, device=DEV)
    L = dgp.lib()
    assert L.dgp_layernorm_backward(None, 0, BF16, None, 0, None, dgp.SCALE_MX128, None, BF16, None, 0, 1e-5, None,
                                    dw.data_ptr(), db.data_ptr(), 0, k, None, 0, stream()) == 0
    assert not bool(dw.any()) and not bool(db.any())
    dw.fill_(7.0)
    assert L.dgp_rmsnorm_backward(None, 0, BF16, None, 0, None, dgp.SCALE_NONE, None, BF16, None, 0, 1e-5, None,
                                  dw.data_ptr(), 0, k, None, 0, stream()) == 0
    assert not bool(dw.any())
