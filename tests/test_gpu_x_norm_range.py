"""GPU tests of rows whose sums leave fp32's range in the layer norm and in the norms' gradients,
as the header describes them."""
import pytest
import torch

import dense_gemm_packer_amd as dgp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rows(k, scale, seed=1):
    """Four rows of fp32: the second and the last of ordinary size."""
    x = torch.randn(4, k, generator=torch.Generator().manual_seed(seed))
    x[[0, 2]] *= scale
    return x.to(DEV)


@pytest.mark.parametrize("k", [512, 4096, 9216])
def test_squares_beyond_the_range(k):
    """xhat is 0: y the bias, dx the residual's gradient; the rows' part of dw is 0."""
    x, dy, r = rows(k, 1e21), rows(k, 1.0, 2), rows(k, 1.0, 3)
    w, b = torch.rand(2, k, generator=torch.Generator().manual_seed(4)).to(DEV)
    y = dgp.layernorm_quantize(x, w, b, dgp.SCALE_NONE)[0]
    assert all(torch.equal(y[i], b.bfloat16()) for i in (0, 2)) and bool(torch.isfinite(y.float()).all())
    for f in (dgp.layernorm_backward, dgp.rmsnorm_backward):
        got = f(dy, x, w, residual_grad=r)
        assert torch.equal(got[0][[0, 2]], r[[0, 2]])
        own = f(dy[[1, 3]], x[[1, 3]], w, residual_grad=r[[1, 3]])
        assert torch.equal(got[0][[1, 3]], own[0])
        assert bool(((got[1] - own[1]).abs() <= 2.0 ** -22 * (dy[1].abs() + dy[3].abs()) * 8).all())


@pytest.mark.parametrize("k", [512, 9216])
def test_sums_beyond_the_range(k):
    """A sum of x (the layer norm's mean), or of its products with g, beyond 3.4e38: NaN in that row."""
    x, dy = rows(k, 1.0), rows(k, 1.0, 2)
    w = torch.ones(k, device=DEV)
    x[0] = 3e38
    assert bool(torch.isnan(dgp.layernorm_quantize(x, w, None, dgp.SCALE_NONE)[0][0].float()).all())
    dx = dgp.layernorm_backward(dy, x, w)[0]
    assert bool(torch.isnan(dx[0]).all()) and bool(torch.isfinite(dx[1:]).all())
    x[0] = 1e30
    dy[0] = 1e10
    dx = dgp.rmsnorm_backward(dy, x, w)[0]
    assert bool(torch.isnan(dx[0]).all()) and bool(torch.isfinite(dx[1:]).all())
