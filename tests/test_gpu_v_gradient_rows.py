"""GPU tests of what a workgroup carries from one step to the next in the norms'
gradients (sums, the row loaded ahead, LDS used in turn), on dense rows, several
steps for every split of a row over waves; of parts of very uneven groups in the
weights' gradients; and of the backward product inside the experts' step."""
import pytest
import torch

import dense_gemm_packer_amd as dgp
from gradient_common import GRAD_MODES, activations, check_near
from operand_common import EPS
from test_gpu_p_norm_gradients import run_norm
from test_gpu_q_wgrad import OUTS, equal, grouped_case
from test_gpu_r_gradient_runs import Layer, check_product, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# rows a step: 256 workgroups of 16, 8, 4, 3, 2 and 1 rows side by side; 1024 workgroups beyond 8192
STEPS = [(13000, 512), (7000, 576), (3100, 2048), (2400, 2112), (1700, 4096), (900, 8192), (2100, 8256)]


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("mode", ["none", "mx128"])
@pytest.mark.parametrize("m,k", STEPS)
def test_three_and_more_steps(layer, mode, m, k):
    if mode != "none":
        k = (k + 127) // 128 * 128
    run_norm(layer, "bf16", "f32", mode, m, k, True, m)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("x_type", ["f32", "f16"])
@pytest.mark.parametrize("m,k", [(2400, 2112), (1700, 4096), (2100, 8256)])
def test_three_and_more_steps_of_other_types(layer, x_type, m, k):
    run_norm(layer, x_type, x_type, "none", m, k, False, m)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("m,k", STEPS)
def test_many_steps_repeat_their_bits(layer, m, k):
    x, dy = activations(m, k, torch.bfloat16, 1).to(DEV), activations(m, k, torch.bfloat16, 2).to(DEV)
    w = torch.ones(k, device=DEV)
    fn = dgp.layernorm_backward if layer else dgp.rmsnorm_backward
    first = fn(dy, x, w, residual_grad=dy)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, fn(dy, x, w, residual_grad=dy)))


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("m,k", STEPS)
def test_a_row_does_not_depend_on_its_place(layer, m, k):
    """dX of rows in another order, in other workgroups and steps: the same bits."""
    x, dy = activations(m, k, torch.bfloat16, 3).to(DEV), activations(m, k, torch.bfloat16, 4).to(DEV)
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    fn = dgp.layernorm_backward if layer else dgp.rmsnorm_backward
    order = torch.randperm(m, generator=torch.Generator().manual_seed(5)).to(DEV)
    assert torch.equal(fn(dy[order], x[order], w)[0], fn(dy, x, w)[0][order])


# ------------------------------------------------ parts of uneven groups

@pytest.mark.parametrize("mode", list(GRAD_MODES))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", list(OUTS))
@pytest.mark.parametrize("counts", [[2000, 5, 300], [0, 2300, 1], [40, 0, 3000], [700, 701, 699]])
def test_parts_of_uneven_groups(mode, gather, out, counts):
    """Several parts a group: some of a short group's hold its last rows, some none."""
    n, k = 144, 256
    kw, want = grouped_case(mode, counts, n, k, gather, 9, sum(counts))
    m = kw["dC"].shape[0]
    assert dgp.lib().dgp_wgrad_workspace_bytes(m, n, k, len(counts)) >= 2 * len(counts) * n * k * 4
    assert equal(dgp.gemm_wgrad(**kw, out_dtype=OUTS[out]), want)
    if out == "f32":
        c = torch.randint(-100, 100, want.shape, generator=torch.Generator().manual_seed(3)).float().to(DEV)
        total = c.cpu().double() + want
        assert dgp.gemm_wgrad(**kw, out=c, accumulate=True) is c
        assert equal(c, total)


# --------------------------------------------------- the experts' step

@pytest.mark.parametrize("mode", ["none", "block128", "mx128"])
@pytest.mark.parametrize("m,k,f,e,x_rows", [(60, 256, 256, 5, 17), (900, 640, 384, 8, 300)])
def test_backward_product_of_experts(mode, m, k, f, e, x_rows):
    """The gradient of the experts' input, by expert, and its sum over each token's rows."""
    l = Layer(mode, k, f, m, 70 + m, e, x_rows)
    o = l.step()
    rows = l.product(o.dC, None, (l.W1.t, None), dgp.SCALE_NONE)
    for i, (lo, hi) in enumerate(zip(l.off.tolist(), l.off.tolist()[1:])):
        if hi > lo:
            check_product(rows[lo:hi], f64(o.dC)[lo:hi], l.W1.tv[i].t(), "none")
    used = l.list.long().cpu()[:m - 8]
    add = lambda t: torch.zeros(x_rows, k, dtype=torch.float64).index_add_(0, used, t)  # noqa: E731
    # (every row of a token adds one rounding to the others)
    most = int(torch.bincount(used).max())
    check_near(o.dA, add(f64(rows)[:m - 8]), EPS * most * add(f64(rows)[:m - 8].abs()), torch.bfloat16)
