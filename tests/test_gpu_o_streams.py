"""GPU tests of the streams that the products take."""
import types

import pytest
import torch

import dense_gemm_packer_amd as dgp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def operands():
    g = torch.Generator().manual_seed(5)
    A = torch.randn(32, 256, generator=g).bfloat16().to(DEV)
    Bs = dgp.preshuffle_b(torch.randn(128, 256, generator=g).bfloat16().to(DEV))
    return A, Bs


def test_a_raw_handle_with_a_given_output():
    """As dgp.preshuffle_b and the split-K products: with `out` given, any object
    that holds a stream's handle names the stream."""
    A, Bs = operands()
    want = dgp.gemm_preshuffle(A, Bs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    got = dgp.gemm_preshuffle(A, Bs, out=out, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    side.synchronize()
    assert got is out and torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_a_raw_handle_without_an_output_is_refused():
    A, Bs = operands()
    with pytest.raises(TypeError, match="torch stream"):
        dgp.gemm_preshuffle(A, Bs, stream=types.SimpleNamespace(cuda_stream=0))
    with pytest.raises(AttributeError, match="cuda_stream"):
        dgp.gemm_preshuffle(A, Bs, out=torch.zeros(32, 128, dtype=torch.bfloat16, device=DEV), stream="s")


@pytest.mark.parametrize("given", [False, True])
def test_torch_streams(given):
    A, Bs = operands()
    want = dgp.gemm_preshuffle(A, Bs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, torch.cuda.ExternalStream(side.cuda_stream), torch.cuda.default_stream()):
        out = torch.zeros_like(want) if given else None
        torch.cuda.synchronize()
        got = dgp.gemm_preshuffle(A, Bs, out=out, stream=s)
        s.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
