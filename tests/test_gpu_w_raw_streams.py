"""GPU tests of streams given as any object with a `cuda_stream` handle: taken where every
output is given and no workspace is needed, refused elsewhere."""
import types

import pytest
import torch

import dense_gemm_packer_amd as dgp
from test_gpu_k_operand_runs import same
from test_gpu_r_gradient_runs import calls

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TAKEN = {0: "layer norm", 3: "gate gradients"}      # of calls(): the others have a workspace


def raw():
    side = torch.cuda.Stream()
    return side, types.SimpleNamespace(cuda_stream=side.cuda_stream)


@pytest.mark.parametrize("i", range(5))
def test_raw_handle(i):
    f, outs = calls()[i]
    f(**outs)
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in outs.items()}
    side, handle = raw()
    for t in outs.values():
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    if i in TAKEN:
        f(stream=handle, **outs)
        side.synchronize()
        assert all(same(outs[n], want[n]) for n in outs)
    else:
        with pytest.raises(TypeError, match="stream must be a torch stream"):
            f(stream=handle, **outs)
    with pytest.raises(TypeError, match="stream must be a torch stream"):      # outputs to allocate
        f(stream=handle)


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_norms_that_have_every_output(norm):
    m, k = 70, 512
    x, r = torch.randn(2, m, k, device=DEV).bfloat16()
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    f = (lambda *a, **kw: dgp.layernorm_quantize(x, w, None, *a, **kw)) if norm == "layer" else \
        (lambda *a, **kw: dgp.rmsnorm_quantize(x, w, *a, **kw))
    want = f(dgp.SCALE_MX128, residual=r)
    outs = dict(zip(("out", "scales", "residual_out"), (torch.empty_like(t) for t in want)))
    torch.cuda.synchronize()
    side, handle = raw()
    f(dgp.SCALE_MX128, residual=r, stream=handle, **outs)
    side.synchronize()
    assert all(same(a, b) for a, b in zip(want, outs.values()))
    for name in outs:                   # one of them to allocate
        with pytest.raises(TypeError, match="stream must be a torch stream"):
            f(dgp.SCALE_MX128, residual=r, stream=handle, **{n: t for n, t in outs.items() if n != name})
    scale = torch.full((1,), 0.01, device=DEV)
    want = f(dgp.SCALE_TENSOR, scale=scale)[0]
    q = torch.empty_like(want)
    torch.cuda.synchronize()
    f(dgp.SCALE_TENSOR, scale=scale, out=q, stream=handle)
    side.synchronize()
    assert same(q, want)
