"""GPU tests of the layer norm and the gradients as a training step uses them:
a gated layer and a layer of experts forward and back, every product and
gradient against 64 bits at the values that it was given; calls of two threads
at once, given streams, graphs replayed in turn with other inputs and eager
work between them, the LDS-poison debug build, and sizes past 32 bits."""
import threading
import types

import pytest
import torch

import dense_gemm_packer_amd as dgp
from gradient_common import (GRAD_MODES, activations, check_near, check_operand_near, kept, kept_values, layernorm_reference,
                             norm_backward_reference, swiglu_backward_reference)
from operand_common import EPS
from test_gpu_j_grouped import aligned_loss
from test_gpu_k_operand_runs import needs, same
from test_gpu_q_wgrad import equal, grads, grouped_case, whole

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
f64 = lambda t: t.cpu().double()  # noqa: E731


# ------------------------------------------------------- a training step

def split(S, mode):
    """The scales of a checkpoint's two halves."""
    if mode == "none":
        return None, None
    k = S.shape[1] // 2
    return S[:, :k], S[:, k:]


def weights(n, k, mode, seed, e=0):
    """A weight as the forward product's operand, its transpose as the backward one's, and both in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    B = (torch.randn(max(e, 1), n, k, generator=g) * k ** -0.5).bfloat16()
    Bt = B.transpose(1, 2).contiguous().to(DEV)
    t = dgp.preshuffle_b(Bt.view(-1, n)).view(Bt.shape)
    if mode == "none":
        s, sB, Bv = dgp.preshuffle_b(B.view(-1, k).to(DEV)).view(B.shape), None, B.double()
    else:
        s, sB = dgp.quantize_b(B.to(DEV), GRAD_MODES[mode])
        codes = dgp.unshuffle_b(s.view(-1, k)).view(s.shape)
        if mode == "mx128":
            Bv = torch.stack([kept_values(c, v, mode) for c, v in zip(codes, sB)])
        else:
            Bv = f64(codes) * f64(sB).repeat_interleave(128, 1).repeat_interleave(128, 2)
    return types.SimpleNamespace(s=s if e else s[0], sB=sB if e or sB is None else sB[0], t=t if e else t[0], v=Bv, tv=B.double())


class Layer:
    """h = x + r, out = W2 (gated activation of W1 norm(h)); e experts where e > 0."""

    def __init__(self, mode, k, f, m, seed, e=0, x_rows=None):
        g = torch.Generator().manual_seed(seed)
        self.mode, self.code, self.f, self.m = mode, GRAD_MODES[mode], f, m
        self.w, self.b = ((c + 0.3 * torch.randn(k, generator=g)).bfloat16().to(DEV) for c in (1, 0))
        self.W1, self.W2 = weights(2 * f, k, mode, seed + 1, e), weights(k, f, mode, seed + 2, e)
        rows = x_rows or m
        self.x, self.r = (activations(rows, k, torch.bfloat16, seed + i).to(DEV) for i in (3, 4))
        self.dout = (1e-2 * activations(m, k, torch.bfloat16, seed + 5).float()).bfloat16().to(DEV)
        self.off = self.list = None
        if e:
            cuts = torch.randint(0, m - 8, (e - 1,), generator=g).sort().values
            cuts[e // 2] = cuts[e // 2 - 1]           # an expert without rows
            self.off = torch.cat([torch.tensor([0]), cuts, torch.tensor([m - 8])]).to(torch.int32).to(DEV)
            self.list = torch.randint(0, rows, (m,), generator=g).to(torch.int32).to(DEV)

    def product(self, A, sA, W, mode, rows=None):
        if self.off is None:
            return dgp.gemm_preshuffle(A, W[0], sA, W[1], scale_mode=mode)
        out = torch.zeros(self.m, W[0].shape[1], dtype=torch.bfloat16, device=DEV)   # (rows of no expert stay)
        return dgp.gemm_preshuffle_grouped(A, W[0], self.off, sA, W[1], mode, rows=rows, out=out)

    def step(self):
        o, f = types.SimpleNamespace(), self.f
        o.A, o.sA, o.h = dgp.layernorm_quantize(self.x, self.w, self.b, self.code, residual=self.r)
        o.C = self.product(o.A, o.sA, (self.W1.s, self.W1.sB), self.code, self.list)
        o.Y, o.sY = dgp.swiglu_quantize(o.C[:, :f], o.C[:, f:], self.code)
        o.out = self.product(o.Y, o.sY, (self.W2.s, self.W2.sB), self.code)
        # what the backward pass keeps besides the operands
        keep = (lambda t: (t, None)) if self.mode == "none" else lambda t: dgp.quantize(t, self.code)
        o.hq, o.hs = keep(o.h)
        o.cq, o.cs = keep(o.C)
        o.dW2 = dgp.gemm_wgrad(self.dout, o.Y, o.sY, self.code, offsets=self.off)
        o.dY = self.product(self.dout, None, (self.W2.t, None), dgp.SCALE_NONE)
        gs, us = split(o.cs, self.mode)
        o.dC = dgp.swiglu_backward(o.dY, o.cq[:, :f], o.cq[:, f:], self.code, gate_scales=gs, up_scales=us)
        o.dW1 = dgp.gemm_wgrad(o.dC, o.A, o.sA, self.code, offsets=self.off, rows=self.list)
        o.dA = self.product(o.dC, None, (self.W1.t, None), dgp.SCALE_NONE)
        if self.off is not None:       # back to the tokens
            o.dA = torch.zeros(self.x.shape, dtype=torch.float32, device=DEV).index_add_(0, self.list.long()[:self.m - 8], o.dA[:self.m - 8].float()).bfloat16()
        res = self.dout if self.off is None else None
        o.dx, o.dw, o.db = dgp.layernorm_backward(o.dA, o.hq, self.w, self.code, scales=o.hs, residual_grad=res)
        return o


def check_product(C, a, b, mode):
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    err = (a.shape[1] + 8) * EPS * size + (aligned_loss(a, b) if mode != "none" else 0)
    check_near(C, want, err, torch.bfloat16)


def check_wgrad(got, d, x, mode):
    """As test_real_values: fp32 sums, block scales to 2^-17 of x."""
    want, size = d.t() @ x, d.abs().t() @ x.abs()
    lost = EPS * (d.shape[0] + 8) + (2.0 ** -17 + EPS if mode == "block128" else 0)
    check_near(got, want, size * lost, torch.float32)


def check_step(l, o):
    mode, f = l.mode, l.f
    h, y, err = layernorm_reference(l.x.cpu(), l.r.cpu(), l.w.cpu(), l.b.cpu(), 1e-5)
    check_near(o.h, h, EPS * h.abs(), torch.bfloat16)
    check_operand_near(o.A, o.sA, y, err, mode)
    A, Y, dC, dout = kept_values(o.A, o.sA, mode), kept_values(o.Y, o.sY, mode), f64(o.dC), f64(l.dout)
    spans = [(0, l.m)] if l.off is None else list(zip(l.off.tolist(), l.off.tolist()[1:]))
    An = A if l.list is None else A[l.list.long().cpu()]
    for e, (lo, hi) in enumerate(spans):
        part = (lambda t: t) if l.off is None else lambda t: t[e]
        check_wgrad(part(o.dW2), dout[lo:hi], Y[lo:hi], mode)
        check_wgrad(part(o.dW1), dC[lo:hi], An[lo:hi], mode)
        if hi > lo:
            check_product(o.C[lo:hi], An[lo:hi], l.W1.v[e], mode)
            check_product(o.out[lo:hi], Y[lo:hi], l.W2.v[e], mode)
            check_product(o.dY[lo:hi], dout[lo:hi], l.W2.tv[e].t(), "none")
            if l.off is None:
                check_product(o.dA, dC, l.W1.tv[e].t(), "none")
    C = kept_values(o.cq, o.cs, mode)
    check_near(o.dC, *swiglu_backward_reference(o.dY.cpu(), C[:, :f], C[:, f:]), torch.bfloat16)
    ref = norm_backward_reference(o.dA.cpu(), kept_values(o.hq, o.hs, mode), l.w.cpu(), l.dout.cpu() if l.off is None else None, 1e-5, True)
    check_near(o.dx, *ref["dx"], torch.bfloat16)
    check_near(o.dw, *ref["dw"], torch.float32)
    check_near(o.db, *ref["db"], torch.float32)


@pytest.mark.parametrize("mode", ["none", "block128", "mx128"])
@pytest.mark.parametrize("m,k,f", [(1, 256, 384), (77, 512, 640), (600, 1152, 512)])
def test_gated_layer(mode, m, k, f):
    l = Layer(mode, k, f, m, 40 + m)
    check_step(l, l.step())


@pytest.mark.parametrize("mode", ["none", "block128", "mx128"])
@pytest.mark.parametrize("m,k,f,e,x_rows", [(60, 256, 256, 5, 17), (900, 640, 384, 8, 300)])
def test_layer_of_experts(mode, m, k, f, e, x_rows):
    l = Layer(mode, k, f, m, 70 + m, e, x_rows)
    check_step(l, l.step())


def test_micro_batches_add_up():
    """Two halves of a batch accumulated are the whole batch's gradient (whole numbers: exactly)."""
    X, S, xv = whole("mx128", 150, 384, 5)
    dY, d = grads(150, 144, 6)
    out = dgp.gemm_wgrad(dY[:70], X[:70], S[:70], dgp.SCALE_MX128)
    dgp.gemm_wgrad(dY[70:], X[70:], S[70:], dgp.SCALE_MX128, out=out, accumulate=True)
    assert equal(out, d.t() @ xv)


# --------------------------------------------------- places and sizes

@pytest.mark.parametrize("k", [256, 8192, 8256, 40960])
@pytest.mark.parametrize("m", [1, 5, 300])
def test_layernorm_onto_its_input(m, k):
    """Q (bf16) in X's own rows and in the residual's, the new stream in the other: also rows read more than once."""
    x, r = (activations(m, k, torch.bfloat16, s, mean=3.0).to(DEV) for s in (81, 82))
    w = torch.full((k,), 0.75, dtype=torch.bfloat16, device=DEV)
    want, _, h = dgp.layernorm_quantize(x, w, w, dgp.SCALE_NONE, residual=r)
    for swap in (False, True):
        x1, r1 = x.clone(), r.clone()
        out, stream = (r1, x1) if swap else (x1, r1)
        Q, _, H = dgp.layernorm_quantize(x1, w, w, dgp.SCALE_NONE, residual=r1, out=out, residual_out=stream)
        assert same(Q, want) and same(H, h) and Q is out and H is stream


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("k", [64, 512, 1280, 8192, 8256, 16448])
@pytest.mark.parametrize("m", [1, 300])
def test_norm_gradient_onto_its_inputs(layer, k, m):
    """dX in the residual gradient's place; where rows are read once, in dY's and in X's."""
    x, dy, r = (activations(m, k, torch.bfloat16, s).to(DEV) for s in (83, 84, 85))
    w = torch.full((k,), 0.75, dtype=torch.bfloat16, device=DEV)
    f = dgp.layernorm_backward if layer else dgp.rmsnorm_backward
    want = f(dy, x, w, residual_grad=r)
    for place in "ryx":
        t = dict(x=x.clone(), y=dy.clone(), r=r.clone())
        call = lambda: f(t["y"], t["x"], w, residual_grad=t["r"], dx=t[place])  # noqa: E731, B023
        if place != "r" and k > 8192:
            with pytest.raises(dgp.DgpError, match="overlap"):
                call()
            continue
        got = call()
        assert got[0] is t[place] and all(same(a, b) for a, b in zip(got, want))
    both = f(dy, x, w, residual_grad=dy)
    t = dy.clone()
    if k <= 8192:                      # one tensor as three
        assert all(same(a, b) for a, b in zip(f(t, x, w, residual_grad=t, dx=t), both))


def test_nothing_to_do():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    assert tuple(dgp.swiglu_backward(z(0, 256), z(0, 256), z(0, 256)).shape) == (0, 512)
    assert tuple(dgp.swiglu_backward(z(4, 0), z(4, 0), z(4, 0)).shape) == (4, 0)
    assert tuple(dgp.layernorm_quantize(z(0, 256), z(256), None, dgp.SCALE_MX128)[0].shape) == (0, 256)
    for f in (dgp.layernorm_backward, dgp.rmsnorm_backward):
        assert tuple(f(z(4, 0), z(4, 0), z(0))[0].shape) == (4, 0)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert tuple(dgp.gemm_wgrad(z(4, 32), z(4, 64), offsets=one).shape) == (0, 32, 64)
    assert tuple(dgp.gemm_wgrad(z(4, 0), z(4, 64)).shape) == (0, 64)
    assert tuple(dgp.gemm_wgrad(z(4, 32), z(4, 0)).shape) == (32, 0)


# -------------------------------------------- threads, streams and graphs

def results(o):
    return [t for t in vars(o).values() if t is not None]


def step_pair():
    return [Layer("mx128", 512, 256, 700, 11), Layer("block128", 512, 256, 90, 12, 4, 50)]


def all_same(a, b):
    return all(same(x, y) for x, y in zip(results(a), results(b), strict=True))


def test_two_threads_on_two_streams():
    layers = [Layer("mx128", 512, 256, 700, 11), Layer("block128", 512, 256, 500, 12)]
    want = [l.step() for l in layers]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got[i] = layers[i].step()
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors
    for g, w in zip(got, want):
        assert all_same(g, w)


def calls():
    """(call, its outputs as keyword arguments) of every operator, with a workspace each."""
    k, m = 512, 900
    x, dy = (activations(m, k, torch.bfloat16, s).to(DEV) for s in (1, 2))
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    Q, S = dgp.quantize(x, dgp.SCALE_MX128)
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
    bf = dict(t=torch.bfloat16)
    return [(lambda **kw: dgp.layernorm_quantize(x, w, w, dgp.SCALE_NONE, **kw), dict(out=e(m, k, **bf))),
            (lambda **kw: dgp.layernorm_backward(dy, x, w, **kw), dict(dx=e(m, k, **bf), dweight=e(k), dbias=e(k))),
            (lambda **kw: dgp.rmsnorm_backward(dy, Q, w, dgp.SCALE_MX128, S, **kw), dict(dx=e(m, k, **bf), dweight=e(k))),
            (lambda **kw: dgp.swiglu_backward(dy, x, x, **kw), dict(out=e(m, 2 * k, **bf))),
            (lambda **kw: dgp.gemm_wgrad(dy, Q, S, dgp.SCALE_MX128, **kw), dict(out=e(k, k)))]


def test_given_streams():
    """A torch stream, with and without outputs; a raw handle with all of them."""
    for f, outs in calls():
        f(**outs)
        torch.cuda.synchronize()
        want = {n: t.clone() for n, t in outs.items()}
        side = torch.cuda.Stream()
        for s in (side, torch.cuda.ExternalStream(side.cuda_stream), types.SimpleNamespace(cuda_stream=side.cuda_stream)):
            for t in outs.values():
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            try:
                f(stream=s, **outs)
            except TypeError:       # a workspace or an output to allocate needs a torch stream
                assert isinstance(s, types.SimpleNamespace)
                continue
            side.synchronize()
            assert all(same(outs[n], want[n]) for n in outs)
        got = f(stream=side)
        side.synchronize()
        got = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
        assert all(same(g, t) for g, t in zip(got, want.values()))


def test_two_graphs_in_turn():
    """Two captured steps, replayed in turn, with eager calls and other inputs between them."""
    layers = step_pair()
    want = [l.step() for l in layers]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for l in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(l.step())
        graphs.append(graph)
    # the scattered sum over experts' rows is torch's, in no fixed order: only what comes before it
    fixed = [lambda o: results(o), lambda o: [o.A, o.C, o.Y, o.out, o.dW2, o.dY, o.dC, o.dW1]]
    for turn in range(4):
        for i in (0, 1):
            graphs[i].replay()
            eager = layers[1 - i].step()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(fixed[i](outs[i]), fixed[i](want[i]))), (turn, i)
            assert all(same(a, b) for a, b in zip(fixed[1 - i](eager), fixed[1 - i](want[1 - i]))), (turn, i)
        for l, seed in zip(layers, (201 + turn, 301 + turn)):
            l.x.copy_(activations(*l.x.shape, torch.bfloat16, seed))
            l.dout.copy_(1e-2 * activations(*l.dout.shape, torch.bfloat16, seed + 50).float())
        want = [l.step() for l in layers]
    graphs[0].replay()
    torch.cuda.synchronize()
    check_step(layers[0], outs[0])


# ------------------------------------------------------------- LDS poison

@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_wgrad_on_poisoned_lds(mode, out):
    """1 to 10 steps of 32 rows in a tile, both tiles, with and without a row list: LDS that no
    copy has filled would give NaN."""
    with dgp.lds_poison_build():
        for m in (1, 32, 33, 64, 95, 128, 160, 200, 310):
            X, S, xv = whole(mode, m, 256, m)
            dY, d = grads(m, 144, 5)
            assert equal(dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], out_dtype=out), d.t() @ xv), m
        X, S, xv = whole(mode, 230, 4096, 1)
        dY, d = grads(230, 4096, 2)
        want = (d.float().to(DEV).t() @ xv.float().to(DEV)).cpu().double()
        assert equal(dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], out_dtype=out), want)
        for counts, n, k in (([1, 0, 33, 70, 160, 300], 144, 384), ([37, 0, 130, 1] * 8, 768, 640)):
            for gather in (False, True):
                kw, want = grouped_case(mode, counts, n, k, gather, 9, 3)
                assert equal(dgp.gemm_wgrad(**kw, out_dtype=out), want), (counts, gather)


def test_step_on_poisoned_lds():
    layers = step_pair()[:1] + [Layer("none", 4352, 256, 70, 13)]
    want = [l.step() for l in layers]
    with dgp.lds_poison_build():
        assert all(all_same(l.step(), w) for l, w in zip(layers, want))


# ------------------------------------------------------ sizes past 32 bits

def at_rows(m, k, at, dtype, seed):
    """[m][k] on the device, zero but for the rows `at`; and those rows."""
    some = activations(len(at), k, dtype, seed)
    x = torch.zeros(m, k, dtype=dtype, device=DEV)
    x[at] = some.to(DEV)
    return x, some


def test_layernorm_of_more_rows_than_a_launch_has_threads_for():
    needs(24)
    k, seam = 64, 2 ** 25
    m = seam + 9
    at = [0, seam - 1, seam, m - 1]
    x, some = at_rows(m, k, at, torch.bfloat16, 5)
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    Q, _ = dgp.layernorm_quantize(x, w, w, dgp.SCALE_NONE)
    _, y, err = layernorm_reference(some, None, w.cpu(), w.cpu(), 1e-5)
    check_near(Q[at], y, err, torch.bfloat16)
    assert bool((Q[1:9] == 1).all())


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("mode", ["none", "mx128"])
@pytest.mark.parametrize("k", [1024, 16512])
def test_norm_gradients_past_4_gib(layer, mode, k):
    """dY, x and dX of more than 4 GiB (2^31 elements) each; sums over rows of which six count."""
    needs(50)
    m = 2 ** 31 // k + 300
    at = [0, 1, 2 ** 30 // k, 2 ** 31 // k - 1, 2 ** 31 // k + 1, m - 1]
    x, xs = at_rows(m, k, at, torch.bfloat16, 6)
    X, S, v = kept(xs, mode, DEV)
    if mode == "none":
        X, S = x, None
    else:
        X, S = dgp.quantize(x, GRAD_MODES[mode])
    dY, dys = at_rows(m, k, at, torch.bfloat16, 7)
    w = torch.ones(k, dtype=torch.bfloat16)
    got = (dgp.layernorm_backward if layer else dgp.rmsnorm_backward)(dY, X, w.to(DEV), GRAD_MODES[mode], scales=S, residual_grad=dY, eps=1e-5)
    ref = norm_backward_reference(dys, v, w, dys, 1e-5, layer)
    check_near(got[0][at], *ref["dx"], torch.bfloat16)
    check_near(got[1], *ref["dw"], torch.float32)
    if layer:
        check_near(got[2], *ref["db"], torch.float32)
    assert not bool(got[0][2:9].any())


@pytest.mark.parametrize("mode", ["none", "mx128"])
def test_gate_gradients_of_more_pieces_than_a_launch_counts(mode):
    """2^31 pieces of 8 elements and more: rows around the seam of two launches, and the last ones."""
    needs(130)
    k, seam = 128, 2 ** 27 - 1
    m = seam + 40
    at = [0, seam - 1, seam, seam + 1, m - 1]
    x, xs = at_rows(m, k, at, torch.bfloat16, 8)
    X, S, v = kept(xs, mode, DEV)
    if mode != "none":
        Q = torch.zeros(m, k, dtype=torch.uint8, device=DEV)
        T = torch.zeros(m, 1, dtype=torch.uint8, device=DEV)
        Q[at], T[at] = X.view(torch.uint8), S
        X, S = Q.view(torch.float8_e4m3fn), T
    else:
        X, S = x, None
    D = dgp.swiglu_backward(x, X, X, GRAD_MODES[mode], gate_scales=S, up_scales=S)
    check_near(D[at], *swiglu_backward_reference(xs, v, v), torch.bfloat16)
    assert not bool(D[1:9].any())


@pytest.mark.parametrize("mode,gather", [("none", False), ("mx128", False), ("block128", False), ("mx128", True), ("none", True)])
def test_wgrad_of_rows_past_4_gib(mode, gather):
    """dC of more than 4 GiB, x of more than (with a list: almost) that, a group border on each side."""
    needs(30)
    n, k = 1024, 1024 if mode == "none" else 2048
    m = 2 ** 21 + 300
    xr = m if not gather else (0xFF000000 // (k * (2 if mode == "none" else 1)))
    offsets = [5, 2 ** 20 + 3, 2 ** 21 + 7, m - 9]
    at = [5, 6, 2 ** 20 + 2, 2 ** 20 + 3, 2 ** 20 + 500, 2 ** 21 - 1, 2 ** 21, 2 ** 21 + 6, 2 ** 21 + 7, m - 11, m - 10]
    outside = [0, 4, m - 9, m - 1]
    dY = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
    small, d = grads(len(at), n, 3)
    dY[at] = small
    dY[outside] = float("nan")
    names = list(at) if not gather else [0, xr - 1, xr // 2, 2 ** 20, 7, 9, xr - 2, 11, xr - 3, 12, 13]
    Xs, Ss, xv = whole(mode, len(at), k, 4)
    X = torch.zeros(xr, k, dtype=torch.bfloat16 if mode == "none" else torch.uint8, device=DEV)
    X[names] = Xs if mode == "none" else Xs.view(torch.uint8)
    S = None
    if mode != "none":
        X = X.view(torch.float8_e4m3fn)
        S = torch.full((xr, k // 128), 127, dtype=torch.uint8, device=DEV) if mode == "mx128" else torch.ones(xr, k // 128, device=DEV)
        S[names] = Ss
    rows = None
    if gather:
        rows = torch.full((m,), xr - 5, dtype=torch.int32, device=DEV)
        rows[at] = torch.tensor(names, dtype=torch.int32, device=DEV)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    got = dgp.gemm_wgrad(dY, X, S, GRAD_MODES[mode], offsets=off, rows=rows)
    at_ = torch.tensor(at)
    want = torch.stack([d[(at_ >= lo) & (at_ < hi)].t() @ xv[(at_ >= lo) & (at_ < hi)] for lo, hi in zip(offsets, offsets[1:])])
    assert equal(got, want)


def test_gradients_of_weights_past_4_gib():
    """The last of a stack of gradients of more than 4 GiB; the others are zeros."""
    needs(20)
    n, k, e = 4096, 4096, 70
    X, S, xv = whole("mx128", 20, k, 5)
    dY, d = grads(20, n, 6)
    off = torch.full((e + 1,), 3, dtype=torch.int32, device=DEV)
    off[-1] = 20
    for t in (torch.float32, torch.bfloat16):
        out = torch.full((e if t == torch.float32 else 2 * e, n, k), 3.0, dtype=t, device=DEV)
        o = off if t == torch.float32 else torch.cat([off[:1].expand(e), off])
        dgp.gemm_wgrad(dY, X, S, dgp.SCALE_MX128, offsets=o.contiguous(), out=out)
        assert equal(out[-1], (d[3:].float().to(DEV).t() @ xv[3:].float().to(DEV)).cpu().double())
        assert not any(bool(out[i].any()) for i in (0, 1, out.shape[0] // 2, out.shape[0] - 2))
        del out
