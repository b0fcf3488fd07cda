"""GPU tests of the gated activation where the gate is far below zero: exp(-g)
reaches the end of fp32's range there, the result g exp(g) u does not."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from operand_common import EPS, MODES, TYPES, check_operand

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# Relative error before the output's rounding.  Near gates as in test_swiglu.
# Far ones: four factors exp(g/4), whose arguments (the product with log2 e, and
# that constant itself) are off by half a step of |g| / 4 log2 e each, ln 2 times
# as much of the factor, and 1 ulp of exp2 each; five products.  2 |g| + 8 half
# steps hold both, as |g| >= 80 of them is more than 4 * 2 + 5 - 8.
def delta(g):
    return g.abs() * EPS * 2 + 8 * EPS


def far(m, k, dt, seed):
    """Gates of -180 to -70 and factors that bring the result back to where the
    type's values live: 2^-20 to 2^20 where u can, else u's largest."""
    g = torch.Generator().manual_seed(seed)
    gate = (-180 + 110 * torch.rand(m, k, generator=g, dtype=torch.float64)).to(dt)
    top = min(float(torch.finfo(dt).max), 3e38) / 2
    want = torch.exp2(40 * torch.rand(m, k, generator=g, dtype=torch.float64) - 20)
    gd = gate.double()
    up = torch.clamp(want / (gd * torch.sigmoid(gd)).abs(), max=top)
    up = up * torch.where(torch.rand(m, k, generator=g) < 0.5, -1.0, 1.0)
    return gate, up.to(dt)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("m,k", [(1, 256), (37, 768)])
def test_far_gates(x_type, mode, m, k):
    g, u = far(m, k, TYPES[x_type], 91)
    scale = torch.full((1,), 0.3, device=DEV) if mode == "tensor" else None
    Q, S = dgp.swiglu_quantize(g.to(DEV), u.to(DEV), MODES[mode], scale=scale)
    gd = g.double()
    check_operand(Q, S, gd * torch.sigmoid(gd) * u.double(), mode, delta(gd), scale)


@pytest.mark.parametrize("gate", [-79.5, -80.5, -87.25, -87.5, -88.5, -89.0, -104.0, -120.0, -178.0])
def test_one_far_gate(gate):
    """fp32: 1 + exp(-g) is above 2^126 from about -87.3 on and infinite from -88.7 on."""
    g, u = torch.full((1, 256), gate), torch.full((1, 256), 2e38)
    Q, _ = dgp.swiglu_quantize(g.to(DEV), u.to(DEV), dgp.SCALE_NONE)
    gd = g.double()
    check_operand(Q, None, gd * torch.sigmoid(gd) * u.double(), "none", delta(gd))
    assert bool((Q < 0).all())


@pytest.mark.parametrize("x_type", list(TYPES))
def test_a_far_gate_leaves_its_neighbours_as_they_are(x_type):
    """The bits of a value do not depend on other gates of the call."""
    gen = torch.Generator().manual_seed(93)
    g = (4 * torch.randn(16, 512, generator=gen)).to(TYPES[x_type])
    u = torch.randn(16, 512, generator=gen).to(TYPES[x_type])
    want, _ = dgp.swiglu_quantize(g.to(DEV), u.to(DEV), dgp.SCALE_NONE)
    at = torch.rand(16, 512, generator=gen) < 0.05
    mixed = torch.where(at, torch.full_like(g, -100.0), g)
    got, _ = dgp.swiglu_quantize(mixed.to(DEV), u.to(DEV), dgp.SCALE_NONE)
    keep = ~at
    assert torch.equal(got.cpu()[keep].view(torch.int16), want.cpu()[keep].view(torch.int16))


def test_gates_at_the_ends():
    """Infinities and NaN as the definition has them: -inf / (1 + inf) is a NaN,
    far below -180 the result is -0 or 0, above it is g u."""
    g = torch.tensor([-float("inf"), float("inf"), float("nan"), -1000.0, -3e38, 200.0, 3e38, 0.0] * 32).view(1, 256)
    u = torch.full((1, 256), 0.5)
    Q, _ = dgp.swiglu_quantize(g.to(DEV), u.to(DEV), dgp.SCALE_NONE)
    got = Q.cpu()[0, :8].float().tolist()
    assert got[0] != got[0] and got[1] == float("inf") and got[2] != got[2]
    assert got[3] == 0 and got[4] == 0 and got[5] == 100.0 and abs(got[6] / 1.5e38 - 1) <= 2.0 ** -8 and got[7] == 0
