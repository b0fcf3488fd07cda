"""GPU tests of the gated activation's gradients in fp32: their error is a number of
half steps that does not grow with the gate."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from gradient_common import check_near
from operand_common import EPS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def reference(dy, gate, up):
    """([dg | du], error) at 64-bit values of fp32 numbers.  In half steps, e = exp(-g): the
    exponential instruction 2 (a whole step), its correction 1; s = 1 / (1 + e): 3 of e, the sum 1
    and the reciprocal 2; dy s one more, du another: 8.  e s: 3 of e that 1 + e takes back in part,
    with the reciprocal, the sum and the product 7; so 7 of |dy u s g (1 - s)|, and of
    |dy u s (1 + g (1 - s))| 8 of dy s u, the sum and the product: 10.  Below -80 four factors of 3
    each, six products, a sum: 19.  Below the normal range half a step there for each product."""
    dy, gate, up = dy.double(), gate.double(), up.double()
    s, t = torch.sigmoid(gate), torch.sigmoid(-gate)
    far = gate < -80
    dg, du = dy * up * s * (1 + gate * t), dy * gate * s
    e_dg = torch.where(far, 19 * dg.abs(), 10 * (dy * up * s).abs() * ((gate * t).abs() + (1 + gate * t).abs()))
    return torch.cat([dg, du], -1), EPS * torch.cat([e_dg, torch.where(far, 19, 9) * du.abs()], -1) + 2.0 ** -126


def rows(gates, seed):
    gates = torch.cat([gates, torch.zeros(-gates.numel() % 64)]).view(1, -1)
    g = torch.Generator().manual_seed(seed)
    dy, up = torch.randn(2, 1, gates.shape[1], generator=g)
    return dy, gates, up


@pytest.mark.parametrize("gates", [
    torch.linspace(-110, 110, 20000), torch.linspace(-25, -5, 5000), torch.linspace(-90, -70, 5000), torch.linspace(5, 100, 5000),
    -1.2784645 + torch.linspace(-1e-3, 1e-3, 2000), torch.exp2(torch.linspace(-100, 6, 2000)), -torch.exp2(torch.linspace(-100, 6, 2000)),
], ids=["all", "negative", "far", "positive", "zero of the derivative", "small", "small negative"])
def test_error_does_not_grow_with_the_gate(gates):
    dy, g, u = rows(gates, 5)
    D = dgp.swiglu_backward(dy.to(DEV), g.to(DEV), u.to(DEV))
    check_near(D, *reference(dy, g, u), torch.float32)


def test_gates_without_a_gradient():
    """Gates whose exponential is zero or infinite, and the largest numbers."""
    g = torch.tensor([200.0, 201.0, 1e4, 1e30, 3.4e38, -105.0, -500.0, -1e4, -1e30, -3.4e38] * 32).view(1, -1)
    dy, u = torch.ones_like(g), torch.full_like(g, 0.5)
    dg, du = dgp.swiglu_backward(dy.to(DEV), g.to(DEV), u.to(DEV)).cpu().chunk(2, -1)
    assert bool((dg[g > 0] == 0.5).all()) and bool((dg[g < 0].abs() <= 2.0 ** -126).all())
    assert torch.equal(du[g > 0], g[g > 0]) and bool((du[g < 0].abs() <= 2.0 ** -126).all())


@pytest.mark.parametrize("x_type", [torch.bfloat16, torch.float16, torch.float32])
def test_gates_that_are_no_numbers(x_type):
    """What the formula gives in 64 bits: NaN for a NaN; at infinity g (1 - s) is NaN, dy g s infinite."""
    g = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0] * 32).view(1, -1).to(x_type)
    one = torch.ones_like(g).to(DEV)
    dg, du = dgp.swiglu_backward(one, g.to(DEV), one).cpu().chunk(2, -1)
    assert bool(torch.isnan(dg.view(-1, 4)[:, :3]).all()) and bool(torch.isfinite(dg.view(-1, 4)[:, 3]).all())
    assert bool(torch.isnan(du.view(-1, 4)[:, [0, 2]]).all()) and bool((du.view(-1, 4)[:, 1] == float("inf")).all())
    assert bool(torch.isfinite(du.view(-1, 4)[:, 3]).all())
