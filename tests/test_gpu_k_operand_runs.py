"""GPU tests of the operand operators and the grouped product as a program uses
them: updates in place, sizes past 32 bits, calls of two threads at once,
graphs that are replayed in turn, and the LDS-poison debug build."""
import threading

import pytest
import torch

import dense_gemm_packer_amd as dgp
from operand_common import EPS, MODES, check_operand, dequantize
from test_gpu_i_quantize import norm_delta, norm_reference, rows
from test_gpu_j_grouped import E4M3, TILES, aligned_loss, check, config, operands, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def needs(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


# ------------------------------------------------------------- in place

@pytest.mark.parametrize("m", [3, 700])
@pytest.mark.parametrize("k", [256, 2048, 7168, 40960])
def test_norm_onto_its_input(m, k):
    """Q (bf16) in X's own rows, and in the residual's."""
    if m * k > 1 << 24:
        m = 300
    x = rows(m, k, torch.bfloat16, 81, spread=1.0).to(DEV)
    r = rows(m, k, torch.bfloat16, 82, spread=1.0).to(DEV)
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    want, _, h = dgp.rmsnorm_quantize(x, w, dgp.SCALE_NONE, residual=r)
    x1, r1 = x.clone(), r.clone()
    Q, _, H = dgp.rmsnorm_quantize(x1, w, dgp.SCALE_NONE, residual=r1, out=x1, residual_out=r1)
    assert same(Q, want) and same(H, h) and Q is x1 and H is r1
    x1, r1 = x.clone(), r.clone()
    Q, _, H = dgp.rmsnorm_quantize(x1, w, dgp.SCALE_NONE, residual=r1, out=r1, residual_out=x1)
    assert same(Q, want) and same(H, h)


def test_gate_onto_its_input():
    g = rows(70, 512, torch.bfloat16, 83).to(DEV)
    u = rows(70, 512, torch.bfloat16, 84).to(DEV)
    want, _ = dgp.swiglu_quantize(g, u, dgp.SCALE_NONE)
    for place in (0, 1):
        pair = [g.clone(), u.clone()]
        Q, _ = dgp.swiglu_quantize(pair[0], pair[1], dgp.SCALE_NONE, out=pair[place])
        assert same(Q, want)


@pytest.mark.parametrize("mode", ["tensor", "block128", "mx128", "mx32"])
def test_outputs_right_beside_the_input(mode):
    """Codes and scales in one buffer with the input, on either side of it."""
    e, n, k = 2, 128, 512
    b = rows(e * n, k, torch.bfloat16, 80).to(DEV).view(e, n, k)
    wq, ws = dgp.quantize_b(b, MODES[mode])
    nq, ns, nb = (t.numel() * t.element_size() for t in (wq, ws, b))
    pad = -ns % 16
    buf = torch.zeros(nq + pad + ns + nb + nq + ns, dtype=torch.uint8, device=DEV)
    start = nq + pad + ns
    inside = buf[start:start + nb].view(torch.bfloat16).view(e, n, k)
    inside.copy_(b)
    for q0, s0 in ((0, nq + pad), (start + nb, start + nb + nq)):
        q = buf[q0:q0 + nq].view(wq.dtype).view(wq.shape)
        s = buf[s0:s0 + ns].view(ws.dtype).view(ws.shape)
        dgp.quantize_b(inside, MODES[mode], out=q, scales=s)
        assert same(q, wq) and same(s, ws) and same(inside, b)


# ------------------------------------------------------ sizes past 32 bits

def test_more_pieces_than_a_launch_counts():
    """2^31 pieces of 8 elements and more: rows around the seam of two launches,
    and the last ones."""
    needs(60)
    k, seam = 256, 2 ** 31 // 32 - 1
    m = seam + 70
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    at = [0, seam - 2, seam - 1, seam, seam + 1, m - 1]
    some = rows(len(at), k, torch.bfloat16, 85)
    x[at] = some.to(DEV)
    Q, S = dgp.quantize(x, dgp.SCALE_MX32)
    del x
    q = torch.stack([Q.view(torch.uint8)[i] for i in at]).view(Q.dtype)
    check_operand(q, torch.stack([S[i] for i in at]), some, "mx32")
    assert int(torch.count_nonzero(S)) <= len(at) * (k // 32)


def test_norm_of_more_rows_than_a_launch_has_threads_for():
    """64 threads a row: 2^25 rows to a launch of 2^31 threads."""
    needs(30)
    k, seam = 64, 2 ** 25
    m = 2 * seam + 9
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    at = [0, seam - 1, seam, 2 * seam - 1, 2 * seam, m - 1]
    g = torch.Generator().manual_seed(86)
    some = torch.randn(len(at), k, generator=g).bfloat16()
    x[at] = some.to(DEV)
    w = (1 + 0.2 * torch.randn(k, generator=g)).bfloat16()
    Q, _, H = dgp.rmsnorm_quantize(x, w.to(DEV), dgp.SCALE_NONE, residual=x)
    check_operand(Q[at], None, norm_reference(some, some, w, 1e-6)[1], "none", norm_delta(k))
    assert same(H[at].cpu(), some * 2)


@pytest.mark.parametrize("mode,tile", [("none", None), ("none", (64, 64)), ("none", (16, 64)), ("mx128", None), ("mx128", (64, 256))])
def test_rows_past_4_gib(mode, tile):
    """A and C of more than 4 GiB each; an expert border on each side of them."""
    needs(40)
    k, n, e = (1024 if mode == "none" else 2048), 1024, 3
    m = 2 ** 21 + 300
    _, _, Bs, sB, _, bd = operands(mode, 1, e, n, k, 87)
    g = torch.Generator(device=DEV).manual_seed(88)
    x = torch.randn(m, k, generator=g, device=DEV, dtype=torch.bfloat16)
    A, sA = (x, None) if mode == "none" else dgp.quantize(x, MODES[mode])
    offsets = [5, 2 ** 20 + 3, 2 ** 21 + 7, m - 9]
    out = torch.full((m, n), 3.0, dtype=torch.bfloat16, device=DEV)
    dgp.gemm_preshuffle_grouped(A, Bs, torch.tensor(offsets, dtype=torch.int32, device=DEV), sA, sB, MODES[mode], out=out,
                                config=config(tile))
    assert bool((out[:5] == 3.0).all()) and bool((out[m - 9:] == 3.0).all())
    for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        at = [lo, lo + 1, (lo + hi) // 2, hi - 2, hi - 1]
        a = dequantize(A[at] if mode == "none" else A.view(torch.uint8)[at].view(A.dtype), None if sA is None else sA[at], mode)
        check(out[at], out[at].cpu(), a, bd[i:i + 1], [0, 5], None, k, aligned_loss if mode in E4M3 else None)


@pytest.mark.parametrize("mode,tile", [("none", None), ("tensor", (16, 32)), ("mx32", (64, 128))])
def test_weights_past_4_gib(mode, tile):
    """The last of a stack of weights of more than 4 GiB."""
    needs(60)
    n, k = 4096, 4096
    e = {"none": 140, "tensor": 270, "mx32": 530}[mode]
    A, sA, B1, s1, ad, bd = operands(mode, 20, 1, n, k, 89)
    Bs = torch.zeros((e,) + tuple(B1.shape[1:]), dtype=torch.uint8 if mode != "none" else B1.dtype, device=DEV)
    Bs[-1] = B1[0].view(Bs.dtype)
    sB = None
    if s1 is not None:
        sB = torch.zeros((e,) + tuple(s1.shape[1:]), dtype=s1.dtype, device=DEV)
        sB[-1] = s1[0]
    off = torch.full((e + 1,), 3, dtype=torch.int32, device=DEV)
    off[-1] = 20
    out = torch.full((20, n), 3.0, dtype=torch.bfloat16, device=DEV)
    dgp.gemm_preshuffle_grouped(A, Bs.view(B1.dtype), off, sA, sB, MODES[mode], out=out, config=config(tile))
    before = torch.full((20, n), 3.0, dtype=torch.bfloat16)
    check(out, before, ad, bd, [3, 20], None, k, aligned_loss if mode in E4M3 else None)


# -------------------------------------------- threads, streams and graphs

def chain(x, r, w, Bs, sB, off):
    """Norm, product by expert, gated activation; and a per-tensor quantisation in two launches."""
    A, sA, H = dgp.rmsnorm_quantize(x, w, dgp.SCALE_MX128, residual=r)
    C = dgp.gemm_preshuffle_grouped(A, Bs, off, sA, sB, dgp.SCALE_MX128)
    Q, S = dgp.swiglu_quantize(C[:, :128], C[:, 128:], dgp.SCALE_BLOCK128)
    T, t = dgp.quantize(x, dgp.SCALE_TENSOR)
    return A, sA, H, C, Q, S, T, t


def chain_inputs(seed, m=160, k=512):
    _, _, Bs, sB, _, _ = operands("mx128", 1, 3, 256, k, seed)
    x, r = (rows(m, k, torch.bfloat16, seed + i, spread=1.0).to(DEV) for i in (1, 2))
    off = torch.tensor([0, seed % 100, 110, m], dtype=torch.int32, device=DEV)
    return x, r, torch.ones(k, dtype=torch.bfloat16, device=DEV), Bs, sB, off


def test_two_threads_on_two_streams():
    sets = [chain_inputs(s) for s in (91, 1095)]
    want = [chain(*s) for s in sets]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got[i] = chain(*sets[i])
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
        assert all(same(a, b) for a, b in zip(g, w))


def test_two_graphs_in_turn():
    """Two captures of the chain, replayed in turn, with eager calls between them."""
    sets = [chain_inputs(s) for s in (97, 1099)]
    want = [chain(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(chain(*s))
        graphs.append(graph)
    for turn in range(3):
        for i in (0, 1):
            graphs[i].replay()
            eager = chain(*sets[1 - i])
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(outs[i], want[i])), (turn, i)
            assert all(same(a, b) for a, b in zip(eager, want[1 - i])), (turn, i)
        # other inputs in the same places
        for s, seed in zip(sets, (201 + turn, 301 + turn)):
            s[0].copy_(rows(160, 512, torch.bfloat16, seed, spread=1.0))
        want = [chain(*s) for s in sets]


def test_two_graphs_of_weight_quantisation():
    """The per-tensor form of quantize_b: its largest-magnitude pass lies in the graph."""
    b = torch.randn(3, 256, 1024, generator=torch.Generator().manual_seed(5)).to(DEV)
    graph = torch.cuda.CUDAGraph()
    dgp.quantize_b(b, dgp.SCALE_TENSOR)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        Q, S = dgp.quantize_b(b, dgp.SCALE_TENSOR)
    for seed in (6, 7, 8):
        b.copy_(torch.randn(3, 256, 1024, generator=torch.Generator().manual_seed(seed)) * seed)
        wq, ws = dgp.quantize_b(b, dgp.SCALE_TENSOR)
        graph.replay()
        torch.cuda.synchronize()
        assert same(Q, wq) and same(S, ws)


# ------------------------------------------------------------- LDS poison

@pytest.mark.parametrize("mode", list(MODES))
def test_every_grouped_tile_on_poisoned_lds(mode):
    """1, 2, 3, 5 and 9 k-tiles on every tile (see test_gpu_h_lds_poison.py): a
    read of LDS that no copy has filled gives NaN or -6."""
    per = {"none": 64, "mx32": 256}.get(mode, 128)
    with dgp.lds_poison_build():
        for tile in TILES[mode]:
            for tiles in (1, 2, 3, 5, 9):
                run(mode, [70, 0, 5, 260], 384, per * tiles, 51, tile, gather=tiles % 2 == 0)
        run(mode, [3, 0, 30], 256, per * 28, 53, (16, 64), gather=True)
