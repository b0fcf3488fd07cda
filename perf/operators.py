"""Cases of the operators around the preshuffled-B product: operand quantisation (activations and weights), the
root-mean-square norm and the gated activation that write a quantised operand, and the product grouped by expert.

Every case runs in a plain form (elementary torch operations in 32 bits) and, where `own` is true, through the
library's entry points.  Modes are the library's scale modes:

  none      bf16, no scales
  tensor    e4m3, one fp32 scale s = max(amax / 448, 2^-126) for the matrix (given, for the row operators)
  block128  e4m3, such a scale per row and 128 columns (weights: per 128 x 128)
  mx128     e4m3, one E8M0 byte per row and 128 columns: the smallest power of two with amax <= 448 * scale
  mx32      E2M1, one E8M0 byte per row and 32 columns: 2^(floor(log2 amax) - 2), codes saturating at 6

E8M0 bytes come back as the powers of two that they stand for.  E2M1 codes are taken through a product, so what comes
back is its bf16 result.
"""
import functools

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BITS = {"none": 16, "tensor": 8, "block128": 8, "mx128": 8, "mx32": 4}
STEP = {"none": 64, "tensor": 128, "block128": 128, "mx128": 128, "mx32": 256}   # K is a multiple of this
TOP = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 16 sequences: an activation to 4 bits and its product with a narrow projection
        dict(name="quantize mx32 + product, decode", op="quantize", mode="mx32", x="bf16", m=16, k=7168, n=2048),
        # a prompt's activations with a scale per row and 128 columns
        dict(name="quantize block128, prompt", op="quantize", mode="block128", x="bf16", m=4096, k=8192, n=0),
        # a wide projection's fp32 master weight laid out for the product, once per load or update
        dict(name="quantize_b mx128, weight", op="quantize_b", mode="mx128", x="f32", e=1, n=16384, k=7168),
        # one token: the norm in front of a projection, with the residual stream's update
        dict(name="rmsnorm mx128, token", op="rmsnorm", mode="mx128", x="bf16", w="bf16", m=1, k=7168, res=True),
        # the same for a prompt
        dict(name="rmsnorm block128, prompt", op="rmsnorm", mode="block128", x="bf16", w="bf16", m=4096, k=8192, res=True),
        # an odd batch in fp16 with fp32 norm weights and an unquantised output, no residual
        dict(name="rmsnorm bf16 out, odd", op="rmsnorm", mode="none", x="f16", w="f32", m=1237, k=2112, res=False),
        # the hidden rows of a decode batch routed to 8 experts each
        dict(name="swiglu block128, decode", op="swiglu", mode="block128", x="bf16", m=128, k=2048),
        # the hidden rows of a long prompt
        dict(name="swiglu mx128, prompt", op="swiglu", mode="mx128", x="bf16", m=16391, k=2048),
        # one token through 8 of 64 experts: eight weights of 16 bits are read once
        dict(name="grouped bf16, token", op="grouped", mode="none", tokens=1, topk=8, e=64, n=4096, k=7168, gather=True,
             skew=0.5, pad=0),
        # a decode batch of 64: a few rows for each expert
        dict(name="grouped block128, decode", op="grouped", mode="block128", tokens=64, topk=8, e=64, n=4096, k=7168,
             gather=True, skew=0.5, pad=0),
        # a short prompt's second product in 4 bits, about a hundred rows for each expert, some spare rows behind them
        dict(name="grouped mx32, chunk", op="grouped", mode="mx32", tokens=811, topk=4, e=32, n=7168, k=2048,
             gather=False, skew=0.5, pad=37),
        # a long prompt's first product
        dict(name="grouped bf16, prompt", op="grouped", mode="none", tokens=8192, topk=2, e=16, n=4096, k=8192,
             gather=True, skew=0.5, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(np.log2(lo), np.log2(hi))))


def draw(rng):
    op = rng.choice(["quantize", "quantize_b", "rmsnorm", "swiglu", "grouped", "grouped"])
    mode = rng.choice(["none", "tensor", "block128", "mx128", "mx32"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        mode = "tensor" if mode == "none" else mode
        k = STEP[mode] * _log(rng, 1, 8192 // STEP[mode])
        return dict(op=op, mode=mode, x=x, m=_log(rng, 1, 8192), k=k,
                    n=128 * _log(rng, 1, 32) if mode == "mx32" else 0)
    if op == "quantize_b":
        mode = mode if mode in ("tensor", "block128", "mx128") else "mx128"
        return dict(op=op, mode=mode, x=x, e=rng.choice([1, 1, 2, 5]), n=128 * _log(rng, 1, 32),
                    k=128 * _log(rng, 1, 64))
    if op in ("rmsnorm", "swiglu"):
        mode = "mx128" if mode == "mx32" else mode
        case = dict(op=op, mode=mode, x=x, m=_log(rng, 1, 8192), k=STEP[mode] * _log(rng, 1, 8192 // STEP[mode]))
        if op == "rmsnorm":
            case.update(w=rng.choice([x, "f32"]), res=rng.random() < 0.7)
        return case
    topk = rng.choice([1, 2, 4, 8])
    e = max(topk, _log(rng, 1, 64))
    n, k = 128 * _log(rng, 1, 32), STEP[mode] * _log(rng, 2, 8192 // STEP[mode])
    return dict(op=op, mode=mode, tokens=_log(rng, 1, 8192 // topk), topk=topk, e=e, n=n, k=k,
                gather=rng.random() < 0.5, skew=round(rng.uniform(0.0, 1.2), 2), pad=rng.choice([0, 0, 0, 19]))


@functools.lru_cache(maxsize=64)
def _counts(tokens, topk, e, skew):
    """Rows of each expert where every token goes to `topk` different experts, the low-numbered ones more often."""
    rng = np.random.default_rng([tokens, topk, e])
    score = -skew * np.log1p(np.arange(e)) + rng.gumbel(size=(tokens, e))
    took = np.argpartition(-score, topk - 1, axis=1)[:, :topk]
    return tuple(int(v) for v in np.bincount(took.ravel(), minlength=e))


def work(case):
    op, mode = case["op"], case["mode"]
    bits, k = BITS[mode], case["k"]
    scale = {"none": 0.0, "tensor": 0.0, "block128": 4 / 128, "mx128": 1 / 128, "mx32": 1 / 32}[mode]
    if op == "grouped":
        n, counts = case["n"], _counts(case["tokens"], case["topk"], case["e"], case["skew"])
        rows, live = sum(counts), sum(1 for c in counts if c)
        a_rows = case["tokens"] if case["gather"] else rows
        b_scale = scale / 128 if mode == "block128" else scale
        return {"bytes": a_rows * k * (bits / 8 + scale) + live * n * k * (bits / 8 + b_scale) + rows * n * 2,
                "flops": 2.0 * rows * n * k}
    if op == "quantize_b":
        b_scale = scale / 128 if mode == "block128" else scale
        return {"bytes": case["e"] * case["n"] * k * (SIZE[case["x"]] + bits / 8 + b_scale), "flops": 0.0}
    m, size = case["m"], SIZE[case["x"]]
    if op == "quantize":
        n = case["n"]
        if n:   # codes and scales go on to the product: what is kept is its result
            return {"bytes": m * k * size + n * k * (bits / 8 + scale) + m * n * 2, "flops": 2.0 * m * n * k}
        return {"bytes": m * k * (size + bits / 8 + scale), "flops": 0.0}
    if op == "rmsnorm":
        moved = size * (3 if case["res"] else 1)
        return {"bytes": m * k * (moved + bits / 8 + scale) + k * SIZE[case["w"]], "flops": 0.0}
    return {"bytes": m * k * (2 * size + bits / 8 + scale), "flops": 0.0}


# ----------------------------------------------------------------- inputs

def _activations(g, m, k, dtype, scale=1.0):
    """Rows of different size, and a few columns far above the others, as a residual stream has them."""
    v = torch.randn(m, k, generator=g, device=DEV)
    v *= scale * torch.exp(0.5 * torch.randn(m, 1, generator=g, device=DEV))
    v *= torch.where(torch.rand(k, generator=g, device=DEV) < 0.004, 20.0, 1.0)
    return v.to(dtype)


def _swizzle(b):
    """[rows][bytes] -> the preshuffled layout: 1 KiB blocks of 16 rows x 64 bytes, 16-byte pieces row by row."""
    n, kb = b.shape
    return b.view(n // 16, 16, kb // 64, 4, 16).permute(0, 2, 3, 1, 4).contiguous().view(n, kb)


def _pack4(q):
    """E2M1 values -> packed codes, element 2j in the low nibble."""
    a = q.abs()
    code = (2 * a).to(torch.int32)                          # 0, .5, 1, 1.5 -> 0..3
    code = torch.where(a >= 2, (a + 2).to(torch.int32), code)    # 2, 3 -> 4, 5
    code = torch.where(a >= 4, 6 + (a >= 6).to(torch.int32), code)
    code = code + 8 * (q < 0).to(torch.int32)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)


def _operand(x32, mode, weight=False):
    """A quantised operand as a program holds it: (codes, scales)."""
    if mode == "none":
        return x32.to(torch.bfloat16), None
    q, s = _quantize(x32, mode, weight)
    if mode == "mx32":
        return _pack4(q), s
    return q.to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, mode, k = case["op"], case["mode"], case["k"]
    st = {"case": dict(case)}
    if op == "grouped":
        tokens, topk, e, n = case["tokens"], case["topk"], case["e"], case["n"]
        counts = np.array(_counts(tokens, topk, e, case["skew"]))
        counts = counts[np.random.default_rng(seed).permutation(e)]
        rows = int(counts.sum())
        st["most"] = int(counts.max())
        st["live"] = torch.from_numpy(np.flatnonzero(counts)).to(DEV)   # the experts that have rows
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
        a_rows = tokens if case["gather"] else rows + case["pad"]
        st["A"], st["sA"] = _operand(_activations(g, a_rows, k, torch.float32), mode)
        st["rows"] = None
        if case["gather"]:
            which = torch.arange(tokens, device=DEV, dtype=torch.int32).repeat_interleave(topk)
            which = which[torch.randperm(rows, generator=g, device=DEV)]
            st["rows"] = torch.cat([which, torch.zeros(case["pad"], dtype=torch.int32, device=DEV)])
        parts = [_operand(torch.randn(n, k, generator=g, device=DEV) * k ** -0.5, mode, True) for _ in range(e)]
        st["B"] = torch.stack([p[0] for p in parts])
        st["sB"] = None if mode == "none" else torch.stack([p[1] for p in parts])
        flat = st["B"].view(torch.uint8).view(e * n, -1)
        st["Bs"] = _swizzle(flat).view(st["B"].dtype).view(st["B"].shape)
        # rows behind the last expert's keep what they hold
        st["out"] = torch.randn(rows + case["pad"], n, generator=g, device=DEV).to(torch.bfloat16) if case["pad"] else None
        return st
    if op == "quantize_b":
        e, n = case["e"], case["n"]
        w = torch.randn(e, n, k, generator=g, device=DEV)
        w *= 0.02 * torch.exp(0.3 * torch.randn(e, n, 1, generator=g, device=DEV))
        st["X"] = w.to(TYPES[case["x"]])
        return st
    m, dtype = case["m"], TYPES[case["x"]]
    if op == "quantize":
        st["X"] = _activations(g, m, k, dtype)
        if case["n"]:
            B, st["sB"] = _operand(torch.randn(case["n"], k, generator=g, device=DEV) * k ** -0.5, mode, True)
            st["B"], st["Bs"] = B, _swizzle(B)
        return st
    st["scale"] = torch.full((1,), 0.02, device=DEV)
    if op == "rmsnorm":
        st["X"] = _activations(g, m, k, dtype, 0.5)
        st["residual"] = _activations(g, m, k, dtype, 2.0) if case["res"] else None
        st["weight"] = (1 + 0.1 * torch.randn(k, generator=g, device=DEV)).to(TYPES[case["w"]])
        return st
    st["X"] = _activations(g, m, 2 * k, dtype)   # gate and up side by side, as one product leaves them
    return st


# ------------------------------------------------------------- plain form

def _blocks(x, size):
    return x.unflatten(-1, (x.shape[-1] // size, size))


def _power(e):
    """2^(127 - e) for E8M0 bytes e (0..253), exactly."""
    return ((254 - e) << 23).view(torch.float32)


def _e2m1(v):
    a = v.abs()
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
    q = q + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5.0).float()
    return torch.where(v < 0, -q, q)


def _quantize(x32, mode, weight=False, scale=None):
    """x32 [..., K] -> (values on the code grid, scales); E8M0 scales as bytes."""
    if mode == "tensor":
        s = torch.clamp(x32.abs().amax() / TOP, min=2.0 ** -126) if scale is None else scale
        return torch.clamp(x32 * (1.0 / s), -TOP, TOP), s.reshape(1)
    if mode == "block128" and weight:
        n, k = x32.shape
        b = x32.view(n // 128, 128, k // 128, 128)
        s = torch.clamp(b.abs().amax(dim=(1, 3)) / TOP, min=2.0 ** -126)
        return torch.clamp(b * (1.0 / s)[:, None, :, None], -TOP, TOP).view(n, k), s
    b = _blocks(x32, 32 if mode == "mx32" else 128)
    amax = b.abs().amax(dim=-1)
    if mode == "block128":
        s = torch.clamp(amax / TOP, min=2.0 ** -126)
        return torch.clamp(b * (1.0 / s)[..., None], -TOP, TOP).flatten(-2), s
    mant, exp = torch.frexp(amax)                       # amax = mant * 2^exp, mant in [0.5, 1)
    low = exp.to(torch.int32) - 1 + 127 - (2 if mode == "mx32" else 8)
    if mode == "mx128":
        low = low + (mant > 0.875).to(torch.int32)      # 448 = 1.75 * 2^8
    e = torch.where(amax > 0, torch.clamp(low, min=0), torch.zeros_like(low))
    v = b * _power(e)[..., None]
    q = _e2m1(v) if mode == "mx32" else torch.clamp(v, -TOP, TOP)
    return q.flatten(-2), e.to(torch.uint8)


def _outputs(y32, mode, scale=None):
    if mode == "none":
        return [y32.to(torch.bfloat16)]
    q, s = _quantize(y32, mode, scale=scale)
    out = [q.to(torch.float8_e4m3fn)]
    if mode == "mx128":
        out.append(s.view(torch.float8_e8m0fnu))
    elif scale is None:
        out.append(s)
    return out


def _unpack4(codes):
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(torch.int64)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return values[both]


def _values(codes, s, mode, weight=False):
    """An operand's values in 32 bits."""
    if mode == "none":
        return codes.float()
    if mode == "mx32":
        return (_blocks(_unpack4(codes), 32) * (1.0 / _power(s.to(torch.int32)))[..., None]).flatten(-2)
    v = codes.float()
    if mode == "tensor":
        return v * (s[..., None] if s.dim() > 1 else s)
    if mode == "mx128":
        return (_blocks(v, 128) * (1.0 / _power(s.to(torch.int32)))[..., None]).flatten(-2)
    if weight:
        s = s.repeat_interleave(128, dim=-2)
    return (_blocks(v, 128) * s[..., None]).flatten(-2)


def _plain(st):
    case = st["case"]
    op, mode = case["op"], case["mode"]
    if op == "grouped":
        a = _values(st["A"], st["sA"], mode)
        if st["rows"] is not None:
            a = a[st["rows"]]
        off = st["offsets"]
        ids = st["live"]
        at = off[ids, None] + torch.arange(st["most"], device=off.device)
        live = at < off[ids + 1, None]
        at = torch.where(live, at, 0)
        b = _values(st["B"][ids], None if st["sB"] is None else st["sB"][ids], mode, True)
        b = b.transpose(1, 2).contiguous()
        c = torch.bmm(a[at], b)                          # [experts][rows of the largest][n]
        out = st["out"]
        if out is None:
            out = torch.empty(a.shape[0], case["n"], dtype=torch.bfloat16, device=a.device)
        out[at[live]] = c[live].to(torch.bfloat16)
        return [out]
    if op == "quantize_b":
        x = st["X"].float()
        e, n, k = x.shape
        if mode == "tensor":
            s = torch.clamp(x.abs().amax(dim=(1, 2)) / TOP, min=2.0 ** -126)
            q = torch.clamp(x * (1.0 / s)[:, None, None], -TOP, TOP).view(e * n, k)
        else:
            q, s = _quantize(x.view(e * n, k), mode, True)
        bs = _swizzle(q.to(torch.float8_e4m3fn).view(torch.uint8)).view(torch.float8_e4m3fn)
        return [bs.view(e, n, k), s.view(torch.float8_e8m0fnu).view(e, n, -1) if mode == "mx128" else s.view(e, -1)]
    if op == "quantize":
        x = st["X"].float()
        if case["n"]:
            q, e = _quantize(x, mode)
            a = (_blocks(q, 32) * (1.0 / _power(e.to(torch.int32)))[..., None]).flatten(-2)
            return [torch.mm(a, _values(st["B"], st["sB"], mode).t()).to(torch.bfloat16)]
        return _outputs(x, mode)
    scale = st["scale"] if mode == "tensor" else None
    if op == "rmsnorm":
        h = st["X"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        y = h * torch.rsqrt((h * h).mean(dim=-1, keepdim=True) + 1e-6) * st["weight"].float()
        out = _outputs(y, mode, scale)
        return out if st["residual"] is None else out + [h.to(st["X"].dtype)]
    gate, up = st["X"].float().chunk(2, dim=-1)
    return _outputs(gate / (1.0 + torch.exp(-gate)) * up, mode, scale)


# ------------------------------------------------------- the library's calls

def _own(st):
    import dense_gemm_packer_amd as dgp
    case = st["case"]
    op, mode = case["op"], case["mode"]
    code = {"none": dgp.SCALE_NONE, "tensor": dgp.SCALE_TENSOR, "block128": dgp.SCALE_BLOCK128,
            "mx128": dgp.SCALE_MX128, "mx32": dgp.SCALE_MX32}[mode]
    if op == "grouped":
        A, Bs = st["A"], st["Bs"]
        if mode == "mx32":
            A, Bs = A.view(torch.float4_e2m1fn_x2), Bs.view(torch.float4_e2m1fn_x2)
        return [dgp.gemm_preshuffle_grouped(A, Bs, st["offsets"], st["sA"], st["sB"], code, rows=st["rows"],
                                            out=st["out"])]
    if op == "quantize_b":
        bs, s = dgp.quantize_b(st["X"], code)
        e, n = bs.shape[:2]
        return [bs, s.view(torch.float8_e8m0fnu).view(e, n, -1) if mode == "mx128" else s.view(e, -1)]
    if op == "quantize":
        q, s = dgp.quantize(st["X"], code)
        if case["n"]:
            return [dgp.gemm_preshuffle(q, st["Bs"].view(torch.float4_e2m1fn_x2), s, st["sB"], code)]
        return [q, s.view(torch.float8_e8m0fnu) if mode == "mx128" else s]
    scale = st["scale"] if mode == "tensor" else None
    if op == "rmsnorm":
        got = dgp.rmsnorm_quantize(st["X"], st["weight"], code, residual=st["residual"], scale=scale)
        tail = list(got[2:])
    else:
        k = case["k"]
        got = dgp.swiglu_quantize(st["X"][:, :k], st["X"][:, k:], code, scale=scale)
        tail = []
    if mode == "none" or mode == "tensor":
        return [got[0]] + tail
    return [got[0], got[1].view(torch.float8_e8m0fnu) if mode == "mx128" else got[1]] + tail


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ 64 bits

def _pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _grid(v, mantissa, lowest, top):
    """v rounded to nearest even on a small floating-point grid, saturating."""
    e = torch.clamp(torch.frexp(v)[1].to(torch.int64) - 1, min=lowest)
    step = _pow2(e - mantissa)
    return torch.clamp(torch.round(v / step) * step, -top, top)


def _exact_codes(x, mode, weight=False, scale=None):
    """x [M][K] in 64 bits -> (codes' values, scales' values)."""
    m, k = x.shape
    if mode == "tensor":
        s = torch.clamp(x.abs().max() / 448, min=2.0 ** -126).reshape(1) if scale is None else scale.double()
        return _grid(x / s, 3, -6, 448.0), s
    if mode == "block128":
        if weight:
            s = x.abs().reshape(m // 128, 128, k // 128, 128).transpose(1, 2).flatten(2).max(dim=2)[0] / 448
            full = s.repeat_interleave(128, 0)
        else:
            full = s = x.abs().reshape(m, k // 128, 128).max(dim=2)[0] / 448
        return _grid(x / torch.clamp(full, min=2.0 ** -126).repeat_interleave(128, 1), 3, -6, 448.0), s
    size, top = (32, 6.0) if mode == "mx32" else (128, 448.0)
    big = x.abs().reshape(m, k // size, size).max(dim=2)[0]
    e = torch.frexp(big)[1].to(torch.int64) - 1 - (2 if mode == "mx32" else 8)
    if mode == "mx128":
        e = e + (big > 448 * _pow2(torch.clamp(e, min=-200))).to(torch.int64)
    e = torch.where(big > 0, torch.clamp(e, min=-127), -127)
    s = _pow2(e)
    v = x / s.repeat_interleave(size, 1)
    return (_grid(v, 1, 0, top) if mode == "mx32" else _grid(v, 3, -6, top)), s


def _exact_operand(codes, s, mode, weight=False):
    if mode == "mx32":
        nib = codes.to(torch.int64)
        nib = torch.stack((nib % 16, nib // 16), dim=2).flatten(1)
        e, f = (nib % 8) // 2, nib % 2
        v = torch.where(e > 0, (2 + f) * _pow2(e - 2), 0.5 * f) * (1.0 - 2.0 * (nib // 8))
        return v * _pow2(s.to(torch.int64) - 127).repeat_interleave(32, 1)
    v = codes.to(torch.float64)
    if mode == "none":
        return v
    if mode == "mx128":
        return v * _pow2(s.to(torch.int64) - 127).repeat_interleave(128, 1)
    s = s.to(torch.float64)
    if mode == "block128":
        return v * (s.repeat_interleave(128, 0) if weight else s).repeat_interleave(128, 1)
    return v * s


def exact(case, seed):
    st = prepare(case, seed)
    op, mode, k = case["op"], case["mode"], case["k"]
    if op == "grouped":
        off = st["offsets"].tolist()
        a = _exact_operand(st["A"], st["sA"], mode)
        n_rows = off[-1] + case["pad"]
        out = torch.zeros(n_rows, case["n"], dtype=torch.float64, device=DEV)
        if st["out"] is not None:
            out.copy_(st["out"])
        for e in range(case["e"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                mine = a[lo:hi] if st["rows"] is None else a[st["rows"][lo:hi].long()]
                b = _exact_operand(st["B"][e], None if st["sB"] is None else st["sB"][e], mode, True)
                out[lo:hi] = mine @ b.t().contiguous()
        return [out]
    if op == "quantize_b":
        e, n = case["e"], case["n"]
        qs, ss = [], []
        for x in st["X"].double():
            q, s = _exact_codes(x, mode, True)
            # lane order of a 16-row x 64-byte block: 16-byte piece g of row r at piece 16 g + r
            q = q.reshape(n // 16, 16, k // 64, 4, 16).transpose(1, 2).transpose(2, 3).reshape(n, k)
            qs.append(q)
            ss.append(s if mode == "mx128" else s.reshape(-1))
        return [torch.stack(qs), torch.stack(ss)]
    x = st["X"].double()
    if op == "quantize":
        q, s = _exact_codes(x, mode)
        if case["n"]:
            a = q * s.repeat_interleave(32, 1)
            return [a @ _exact_operand(st["B"], st["sB"], mode).t().contiguous()]
        return [q, s]
    tail = []
    if op == "rmsnorm":
        if st["residual"] is not None:
            x = x + st["residual"].double()
            tail = [x]
        y = x / torch.sqrt(x.pow(2).sum(dim=1, keepdim=True) / k + 1e-6) * st["weight"].double()
    else:
        y = x[:, :k] * torch.sigmoid(x[:, :k]) * x[:, k:]
    if mode == "none":
        return [y] + tail
    q, s = _exact_codes(y, mode, scale=st["scale"] if mode == "tensor" else None)
    return [q] + ([] if mode == "tensor" else [s]) + tail
