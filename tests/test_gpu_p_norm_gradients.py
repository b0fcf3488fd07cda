"""GPU tests of the layer norm that writes a product's operand, and of the
gradients of both norms and of the gated activation, from activations and from
their 8-bit checkpoints, against 64-bit references (gradient_common.py)."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from gradient_common import (GRAD_MODES, activations, check_near, check_operand_near, kept, layernorm_reference,
                             norm_backward_reference, swiglu_backward_reference)
from operand_common import MODES, TYPES

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def vectors(k, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(k, generator=g)).to(dtype), (0.5 * torch.randn(k, generator=g)).to(dtype)


def dev(t):
    return None if t is None else t.to(DEV)


# ------------------------------------------------------------- layer norm

@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("m,k", [(1, 256), (3, 512), (37, 1280), (70, 4352), (2, 7168)])
def test_layernorm(x_type, mode, m, k):
    dt = TYPES[x_type]
    x, r = activations(m, k, dt, k + m), activations(m, k, dt, k, mean=0.7)
    w, b = vectors(k, dt, m)
    scale = torch.full((1,), 0.01, device=DEV) if mode == "tensor" else None
    Q, S, H = dgp.layernorm_quantize(dev(x), dev(w), dev(b), MODES[mode], residual=dev(r), scale=scale)
    h, y, err = layernorm_reference(x, r, w, b, 1e-5)
    check_operand_near(Q, S, y, err, mode, scale)
    check_near(H, h, 2.0 ** -24 * h.abs(), dt)


@pytest.mark.parametrize("m,k", [(5, 64), (9001, 960), (8, 2112), (390, 8192), (3, 16448), (3, 32768), (2, 40960)])
@pytest.mark.parametrize("bias", [False, True])
def test_layernorm_lengths(m, k, bias):
    """Every split of a row over threads, and rows longer than the registers hold."""
    x = activations(m, k, torch.bfloat16, k)
    w, b = vectors(k, torch.float32, k)
    b = b if bias else None
    got = dgp.layernorm_quantize(dev(x), dev(w), dev(b), dgp.SCALE_NONE)
    assert len(got) == 2 and got[1] is None
    _, y, err = layernorm_reference(x, None, w, b, 1e-5)
    check_operand_near(got[0], None, y, err, "none")


@pytest.mark.parametrize("x_type,mean", [("bf16", 100.0), ("f32", 1e4), ("f16", -1000.0)])
def test_layernorm_far_from_zero(x_type, mean):
    x = activations(6, 1024, TYPES[x_type], 5, mean=mean)
    w, b = vectors(1024, TYPES[x_type], 6)
    Q, _ = dgp.layernorm_quantize(dev(x), dev(w), dev(b), dgp.SCALE_NONE)
    _, y, err = layernorm_reference(x, None, w, b, 1e-5)
    check_operand_near(Q, None, y, err, "none")


def test_layernorm_equal_values():
    """Rows without any spread: the bias."""
    x = torch.tensor([[0.0], [3.0], [-1e30], [0.1]], dtype=torch.float32).expand(4, 384).contiguous()
    w, b = vectors(384, torch.float32, 1)
    Q, _ = dgp.layernorm_quantize(dev(x), dev(w), dev(b), dgp.SCALE_NONE)
    assert torch.equal(Q.cpu(), b.bfloat16().expand(4, 384))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_layernorm_not_finite(bad):
    x = activations(4, 512, torch.bfloat16, 8)
    x[2, 77] = bad
    w, b = vectors(512, torch.bfloat16, 2)
    Q, S = dgp.layernorm_quantize(dev(x), dev(w), dev(b), dgp.SCALE_BLOCK128)
    assert bool(torch.isnan(S[2]).all()) and bool(torch.isfinite(S[[0, 1, 3]]).all())
    assert bool(torch.isnan(Q[2].float()).all()) and bool(torch.isfinite(Q[[0, 1, 3]].float()).all())


def test_layernorm_strided_and_in_place():
    wide = activations(9, 1536, torch.bfloat16, 3).to(DEV)
    x = wide[:, 512:1024]
    w, b = (v.to(DEV) for v in vectors(512, torch.bfloat16, 4))
    want, _, h = dgp.layernorm_quantize(x.contiguous(), w, b, dgp.SCALE_NONE, residual=x.contiguous())
    got, _, h2 = dgp.layernorm_quantize(x, w, b, dgp.SCALE_NONE, residual=x)
    assert torch.equal(want, got) and torch.equal(h, h2)
    a, r = x.clone(), x.clone()
    got, _, h2 = dgp.layernorm_quantize(a, w, b, dgp.SCALE_NONE, residual=r, out=a, residual_out=r)
    assert got is a and h2 is r and torch.equal(want, a) and torch.equal(h, r)


# --------------------------------------------------------- norm gradients

def run_norm(layer, x_type, w_type, mode, m, k, res, seed, mean=0.0, eps=1e-5):
    dt = TYPES[x_type]
    X, S, xv = kept(activations(m, k, dt, seed, mean=mean), mode, DEV)
    dy = activations(m, k, dt, seed + 1)
    w, _ = vectors(k, TYPES[w_type], seed)
    r = activations(m, k, dt, seed + 2) if res else None
    fn = dgp.layernorm_backward if layer else dgp.rmsnorm_backward
    got = fn(dev(dy), X, dev(w), GRAD_MODES[mode], scales=S, residual_grad=dev(r), eps=eps)
    ref = norm_backward_reference(dy, xv, w, r, eps, layer)
    check_near(got[0], *ref["dx"], dt)
    check_near(got[1], *ref["dw"], torch.float32)
    if layer:
        check_near(got[2], *ref["db"], torch.float32)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("m,k", [(1, 128), (3, 512), (37, 1280), (130, 4096), (5, 7168)])
def test_norm_backward(layer, x_type, mode, m, k):
    run_norm(layer, x_type, x_type, mode, m, k, (m + k) % 3 != 0, k + m)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("m,k", [(1, 64), (2, 64), (5000, 64), (1500, 576), (777, 1088), (1031, 2048), (530, 2112), (600, 8192),
                                 (3, 8256), (70, 16384), (40, 40960), (1, 9216)])
def test_norm_backward_lengths(layer, m, k):
    run_norm(layer, "bf16", "f32", "none", m, k, True, k)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128"])
def test_norm_backward_long_checkpoint(layer, mode):
    run_norm(layer, "bf16", "bf16", mode, 9, 9344, True, 7)


@pytest.mark.parametrize("x_type,mean", [("bf16", 50.0), ("f32", 1e4)])
def test_layernorm_backward_far_from_zero(x_type, mean):
    run_norm(True, x_type, "f32", "none", 20, 1024, False, 9, mean=mean)


@pytest.mark.parametrize("layer", [True, False])
def test_norm_backward_of_no_rows(layer):
    for k in (256, 9216):
        z = torch.zeros(0, k, dtype=torch.bfloat16, device=DEV)
        w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
        out = torch.full((2, k), 7.0, device=DEV)
        fn = dgp.layernorm_backward if layer else dgp.rmsnorm_backward
        kw = dict(dbias=out[1]) if layer else {}
        got = fn(z, z, w, dweight=out[0], **kw)
        assert tuple(got[0].shape) == (0, k) and not bool(out[0].any())
        assert bool((out[1] == (0.0 if layer else 7.0)).all())


def test_norm_backward_against_differences():
    """The gradient of <dy, y> along random directions, by central differences in 64 bits."""
    m, k, eps = 7, 256, 1e-5
    g = torch.Generator().manual_seed(11)
    x, dy, w, b = (torch.randn(*s, generator=g).float() for s in ((m, k), (m, k), (k,), (k,)))
    for layer in (True, False):
        def f(x, w, b):
            d = x - x.mean(-1, keepdim=True) if layer else x
            return (dy.double() * (d / torch.sqrt((d * d).mean(-1, keepdim=True) + eps) * w + b)).sum()
        fn = dgp.layernorm_backward if layer else dgp.rmsnorm_backward
        got = [t.cpu().double() for t in fn(dev(dy), dev(x), dev(w), eps=eps)]
        at = [x.double(), w.double(), b.double()]
        for i, grad in enumerate(got):
            v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
            h = 1e-4
            hi, lo = [list(at), list(at)]
            hi[i], lo[i] = at[i] + h * v, at[i] - h * v
            want = (f(*hi) - f(*lo)) / (2 * h)
            # differences: h^2 times a third derivative of order |v|^3; fp32: 1e-6 of the terms
            assert abs(float((grad * v).sum() - want)) <= 1e-5 * float((grad * v).abs().sum()) + 1e-5


def test_norm_backward_strides_and_places():
    k = 640
    wide = activations(33, 3 * k, torch.bfloat16, 12).to(DEV)
    dy, x, r = wide[:, :k], wide[:, k:2 * k], wide[:, 2 * k:]
    w = vectors(k, torch.bfloat16, 1)[0].to(DEV)
    want = dgp.layernorm_backward(dy.contiguous(), x.contiguous(), w, residual_grad=r.contiguous())
    got = dgp.layernorm_backward(dy, x, w, residual_grad=r)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for place in range(3):      # dx over dy, x and the residual's gradient
        t = [dy.contiguous().clone(), x.contiguous().clone(), r.contiguous().clone()]
        out = dgp.layernorm_backward(t[0], t[1], w, residual_grad=t[2], dx=t[place])
        assert out[0] is t[place]
        for a, b in zip(want, out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("k", [512, 2048, 8192, 9216])
def test_norm_backward_repeats_its_bits(k):
    x, dy = activations(999, k, torch.bfloat16, 1).to(DEV), activations(999, k, torch.bfloat16, 2).to(DEV)
    w = torch.ones(k, device=DEV)
    first = dgp.layernorm_backward(dy, x, w)
    for _ in range(3):
        for a, b in zip(first, dgp.layernorm_backward(dy, x, w)):
            assert torch.equal(a, b)


def test_norm_backward_of_equal_values():
    """Rows without spread: xhat = 0, dx = (g - mean(g)) / sqrt(eps)."""
    k = 256
    x = torch.tensor([[0.0], [2.5], [-300.0]]).expand(3, k).contiguous()
    dy = activations(3, k, torch.float32, 4)
    w = torch.ones(k)
    dx, dw, db = dgp.layernorm_backward(dev(dy), dev(x), dev(w), eps=1e-2)
    g = dy.double()
    check_near(dx, (g - g.mean(-1, keepdim=True)) * 10, 2.0 ** -24 * 10 * 64 * (g.abs() + g.abs().mean(-1, keepdim=True)), torch.float32)
    assert not bool(dw.any())


def test_norm_backward_not_finite_rows_stay_apart():
    x, dy = activations(40, 1024, torch.bfloat16, 3), activations(40, 1024, torch.bfloat16, 4)
    w = torch.ones(1024, dtype=torch.bfloat16, device=DEV)
    clean = dgp.layernorm_backward(dev(dy), dev(x), w)
    x[17, 5] = float("inf")
    dx, dw, db = dgp.layernorm_backward(dev(dy), dev(x), w)
    keep = [i for i in range(40) if i != 17]
    assert torch.equal(dx[keep], clean[0][keep]) and bool(torch.isnan(dx[17].float()).all())
    assert bool(torch.isnan(dw).all()) and torch.equal(db, clean[2])


# ------------------------------------------------------- gated activation

@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("m,k", [(1, 128), (3, 256), (130, 1152), (7, 2048)])
def test_swiglu_backward(x_type, mode, m, k):
    dt = TYPES[x_type]
    X, S, xv = kept(activations(m, 2 * k, dt, k + m, spread=1.5), mode, DEV)
    dy = activations(m, k, dt, k)
    sg, su = (S[:, :k // 128], S[:, k // 128:]) if mode in ("block128", "mx128") else (S, S)
    D = dgp.swiglu_backward(dev(dy), X[:, :k], X[:, k:], GRAD_MODES[mode], gate_scales=sg, up_scales=su)
    check_near(D, *swiglu_backward_reference(dy, xv[:, :k], xv[:, k:]), dt)


@pytest.mark.parametrize("x_type", ["bf16", "f32"])
def test_swiglu_backward_gates(x_type):
    """Gates from far below to far above zero, around the zero of the derivative, and small ones."""
    dt = TYPES[x_type]
    g = torch.cat([torch.linspace(-110, 110, 2000), -80 + torch.linspace(-1, 1, 200), -1.2784645 + torch.linspace(-1e-2, 1e-2, 200),
                   torch.exp2(-torch.linspace(1, 100, 100)), torch.tensor([0.0, -0.0, 1e30, -1e30, 3e4, -3e4])])
    g = torch.cat([g, torch.zeros(-g.numel() % 64)]).view(1, -1).to(dt)
    gen = torch.Generator().manual_seed(3)
    dy, u = (torch.randn(1, g.shape[1], generator=gen).to(dt) for _ in range(2))
    D = dgp.swiglu_backward(dev(dy), dev(g), dev(u))
    want, err = swiglu_backward_reference(dy, g.double(), u.double())
    # (results below the normal range: half a step there for each of the last two products)
    check_near(D, want, err + 2.0 ** -126, dt)


def test_swiglu_backward_against_differences():
    g = torch.Generator().manual_seed(21)
    dy, gate, up = (torch.randn(5, 192, generator=g).float() for _ in range(3))
    D = dgp.swiglu_backward(dev(dy), dev(gate), dev(up)).cpu().double()
    def f(a, b):
        return dy.double() * a * torch.sigmoid(a) * b
    h, a, b = 1e-5, gate.double(), up.double()
    want = torch.cat([(f(a + h, b) - f(a - h, b)) / (2 * h), (f(a, b + h) - f(a, b - h)) / (2 * h)], -1)
    assert bool(((D - want).abs() <= 1e-6 * (1 + want.abs()) + 1e-6 * dy.double().abs().repeat(1, 2) * (1 + up.double().abs().repeat(1, 2))).all())


def test_swiglu_backward_strides_and_places():
    k = 320
    wide = activations(11, 2 * k + 64, torch.bfloat16, 5).to(DEV)
    gu = wide[:, 64:]
    dy = activations(11, 2 * k, torch.bfloat16, 6).to(DEV)[:, k:]
    want = dgp.swiglu_backward(dy.contiguous(), gu[:, :k].contiguous(), gu[:, k:].contiguous())
    assert torch.equal(want, dgp.swiglu_backward(dy, gu[:, :k], gu[:, k:]))
    assert torch.equal(want[:, k:], dgp.swiglu_backward(dy, gu[:, :k], torch.zeros_like(gu[:, k:]))[:, k:])
    c = gu.contiguous()
    assert dgp.swiglu_backward(dy, c[:, :k], c[:, k:], out=c) is c and torch.equal(want, c)
