"""Cases of the training side: the layer norm that writes a product's operand, the gradients of both norms and of the
gated activation, and a weight's gradient, each from 16-bit activations or from their 8-bit checkpoints.

A checkpoint is what `quantize` makes of an activation, so the forward product's own operand serves as one:

  none      the activation itself (a product's operand: bf16)
  tensor    e4m3, one fp32 scale s = max(amax / 448, 2^-126) for the matrix
  block128  e4m3, such a scale per row and 128 columns
  mx128     e4m3, one E8M0 byte per row and 128 columns: the smallest power of two with amax <= 448 * scale

Every gradient is that of the formula at the values which the checkpoint holds.  Every case runs in a plain form
(elementary torch operations in 32 bits) and, where `own` is true, through the library's entry points.
"""
import functools

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
SCALES = {"none": 0.0, "tensor": 0.0, "block128": 4 / 128, "mx128": 1 / 128}   # bytes of scale per element
TOP = 448.0
EPS = {"layernorm": 1e-5, "rmsnorm": 1e-6}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token: the norm in front of a projection, with the residual stream's update
        dict(name="layernorm mx128, token", op="layernorm", mode="mx128", x="bf16", w="bf16", m=1, k=7168, res=True, bias=True),
        # the same for a batch of training sequences
        dict(name="layernorm block128, batch", op="layernorm", mode="block128", x="bf16", w="bf16", m=4096, k=8192, res=True,
             bias=True),
        # an odd batch in fp16 with fp32 norm weights, the activation kept as it is
        dict(name="layernorm_backward, odd", op="layernorm_backward", mode="none", x="f16", w="f32", m=1237, k=2112, res=False),
        # a batch whose residual stream was kept in 8 bits, the stream's own gradient added
        dict(name="layernorm_backward block128, batch", op="layernorm_backward", mode="block128", x="bf16", w="bf16", m=4096,
             k=8192, res=True),
        # a short sequence
        dict(name="rmsnorm_backward, short", op="rmsnorm_backward", mode="none", x="bf16", w="bf16", m=128, k=7168, res=True),
        # many short rows (a norm per head, or a narrow model) from an mxfp8 checkpoint
        dict(name="rmsnorm_backward mx128, narrow rows", op="rmsnorm_backward", mode="mx128", x="bf16", w="bf16", m=16391,
             k=2048, res=True),
        # a short sequence through a gated layer
        dict(name="swiglu_backward, short", op="swiglu_backward", mode="none", x="bf16", m=128, k=2048),
        # a long batch's gate and up kept in mxfp8, side by side as one product left them
        dict(name="swiglu_backward mx128, batch", op="swiglu_backward", mode="mx128", x="bf16", m=16391, k=2048),
        # a few rows only: a weight's gradient that is little more than its own write
        dict(name="wgrad tensor, short", op="wgrad", mode="tensor", m=128, n=2048, k=2048, out="f32"),
        # 16-bit activations, an odd number of rows and a narrow weight, the gradient in bf16
        dict(name="wgrad bf16, odd rows", op="wgrad", mode="none", m=4109, n=2112, k=7168, out="bf16"),
        # a wide projection from the operand that its own forward product took, into an fp32 gradient
        dict(name="wgrad mx128, batch", op="wgrad", mode="mx128", m=8192, n=8192, k=4096, out="f32"),
        # 32 experts' weights, tokens named by a row list, about a thousand rows for each expert
        dict(name="wgrad block128, experts", op="wgrad", mode="block128", tokens=8192, topk=4, e=32, n=4096, k=2048,
             gather=True, skew=0.5, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(np.log2(lo), np.log2(hi))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_backward", "rmsnorm_backward", "swiglu_backward", "wgrad", "wgrad", "wgrad"])
    mode = rng.choice(["none", "tensor", "block128", "mx128"])
    step = 64 if mode == "none" else 128
    if op != "wgrad":
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        case = dict(op=op, mode=mode, x=x, m=_log(rng, 1, 8192), k=step * _log(rng, 1, 8192 // step))
        if op != "swiglu_backward":
            case.update(w=rng.choice([x, "f32"]), res=rng.random() < 0.7)
        if op == "layernorm":
            case["bias"] = rng.random() < 0.7
        elif rng.random() < 0.2:        # many short rows
            case.update(m=_log(rng, 4096, 65536), k=step * rng.choice([1, 2, 4]))
        case["m"] = min(case["m"], 2 ** 26 // (case["k"] * SIZE[x]))
        return case
    n, k = 16 * _log(rng, 1, 512), step * _log(rng, 1, 8192 // step)
    rows = min(_log(rng, 1, 16384), int(2.5e11 / (n * k)))
    case = dict(op=op, mode=mode, n=n, k=k, out=rng.choice(["f32", "bf16"]))
    if rng.random() < 0.5:
        return dict(case, m=rows)
    topk = rng.choice([1, 2, 4])
    e = max(topk, min(_log(rng, 1, 64), int(2 ** 28 / (n * k))))
    return dict(case, tokens=max(1, rows // topk), topk=topk, e=e, gather=rng.random() < 0.5, skew=round(rng.uniform(0.0, 1.2), 2))


@functools.lru_cache(maxsize=64)
def _counts(tokens, topk, e, skew):
    """Rows of each expert where every token goes to `topk` different experts, the low-numbered ones more often."""
    rng = np.random.default_rng([tokens, topk, e])
    score = -skew * np.log1p(np.arange(e)) + rng.gumbel(size=(tokens, e))
    took = np.argpartition(-score, topk - 1, axis=1)[:, :topk]
    return tuple(int(v) for v in np.bincount(took.ravel(), minlength=e))


def work(case):
    op, mode, k = case["op"], case["mode"], case["k"]
    kept = 1 if mode != "none" else 2 if op == "wgrad" else SIZE[case["x"]]     # bytes of a kept element
    kept += SCALES[mode]
    if op == "wgrad":
        n, e = case["n"], case.get("e", 1)
        rows = case["m"] if "m" in case else case["tokens"] * case["topk"]
        x_rows = case["tokens"] if case.get("gather") else rows
        return {"bytes": rows * n * 2 + x_rows * k * kept + e * n * k * SIZE[case["out"]], "flops": 2.0 * rows * n * k}
    m, size = case["m"], SIZE[case["x"]]
    if op == "swiglu_backward":
        return {"bytes": m * k * (size + 2 * kept + 2 * size), "flops": 0.0}
    if op == "layernorm":
        written = 2 if mode == "none" else 1 + SCALES[mode]
        return {"bytes": m * k * (size * (3 if case["res"] else 1) + written) + k * SIZE[case["w"]] * (2 if case["bias"] else 1),
                "flops": 0.0}
    sums = 2 if op == "layernorm_backward" else 1
    return {"bytes": m * k * (size * (3 if case["res"] else 2) + kept) + k * (SIZE[case["w"]] + 4 * sums), "flops": 0.0}


# ----------------------------------------------------------------- inputs

def _activations(g, m, k, scale=1.0):
    """Rows of different size, and a few columns far above the others, as a residual stream has them."""
    v = torch.randn(m, k, generator=g, device=DEV)
    v *= scale * torch.exp(0.5 * torch.randn(m, 1, generator=g, device=DEV))
    v *= torch.where(torch.rand(k, generator=g, device=DEV) < 0.004, 20.0, 1.0)
    return v


def _gradients(g, m, k, dtype):
    """Small, and of different size from row to row; fp16 ones under a loss scale of 1024."""
    v = torch.randn(m, k, generator=g, device=DEV)
    v *= 1e-3 * torch.exp(0.7 * torch.randn(m, 1, generator=g, device=DEV))
    if dtype == torch.float16:
        v *= 1024
    return v.to(dtype)


def _kept(v, mode, dtype):
    """An activation as the forward pass keeps it: (values or codes, scales)."""
    if mode == "none":
        return v.to(dtype), None
    q, s = _quantize(v.to(dtype).float(), mode)
    return q.to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, mode, k = case["op"], case["mode"], case["k"]
    st = {"case": dict(case)}
    if op == "wgrad":
        n = case["n"]
        if "m" in case:
            rows = x_rows = case["m"]
        else:
            tokens, topk, e = case["tokens"], case["topk"], case["e"]
            counts = np.array(_counts(tokens, topk, e, case["skew"]))[np.random.default_rng(seed).permutation(e)]
            rows = int(counts.sum())
            x_rows = tokens if case["gather"] else rows
            st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
            st["counts"] = [int(c) for c in counts]
            if case["gather"]:
                which = torch.arange(tokens, device=DEV, dtype=torch.int32).repeat_interleave(topk)
                st["rows"] = which[torch.randperm(rows, generator=g, device=DEV)]
        st["X"], st["sX"] = _kept(_activations(g, x_rows, k), mode, torch.bfloat16)
        st["dY"] = _gradients(g, rows, n, torch.bfloat16)
        return st
    m, dtype = case["m"], TYPES[case["x"]]
    if op == "swiglu_backward":
        st["X"], st["sX"] = _kept(_activations(g, m, 2 * k), mode, dtype)     # gate and up side by side
        st["dY"] = _gradients(g, m, k, dtype)
        return st
    st["weight"] = (1 + 0.1 * torch.randn(k, generator=g, device=DEV)).to(TYPES[case["w"]])
    mean = 0.3 * torch.randn(m, 1, generator=g, device=DEV)
    if op == "layernorm":
        st["X"] = (_activations(g, m, k, 0.5) + mean).to(dtype)
        st["residual"] = _activations(g, m, k, 2.0).to(dtype) if case["res"] else None
        st["bias"] = (0.1 * torch.randn(k, generator=g, device=DEV)).to(TYPES[case["w"]]) if case["bias"] else None
        st["scale"] = torch.full((1,), 0.02, device=DEV)
        return st
    st["X"], st["sX"] = _kept(_activations(g, m, k, 2.0) + mean, mode, dtype)
    st["dY"] = _gradients(g, m, k, dtype)
    st["residual"] = _gradients(g, m, k, dtype) if case["res"] else None
    return st


# ------------------------------------------------------------- plain form

def _blocks(x):
    return x.unflatten(-1, (x.shape[-1] // 128, 128))


def _power(e):
    """2^(127 - e) for E8M0 bytes e (0..253), exactly."""
    return ((254 - e) << 23).view(torch.float32)


def _quantize(x32, mode, scale=None):
    """x32 [..., K] -> (values on the e4m3 grid, scales); E8M0 scales as bytes."""
    if mode == "tensor":
        s = torch.clamp(x32.abs().amax() / TOP, min=2.0 ** -126) if scale is None else scale
        return torch.clamp(x32 * (1.0 / s), -TOP, TOP), s.reshape(1)
    b = _blocks(x32)
    amax = b.abs().amax(dim=-1)
    if mode == "block128":
        s = torch.clamp(amax / TOP, min=2.0 ** -126)
        return torch.clamp(b * (1.0 / s)[..., None], -TOP, TOP).flatten(-2), s
    mant, exp = torch.frexp(amax)                       # amax = mant * 2^exp, mant in [0.5, 1)
    low = exp.to(torch.int32) - 1 + 127 - 8 + (mant > 0.875).to(torch.int32)      # 448 = 1.75 * 2^8
    e = torch.where(amax > 0, torch.clamp(low, min=0), torch.zeros_like(low))
    return torch.clamp(b * _power(e)[..., None], -TOP, TOP).flatten(-2), e.to(torch.uint8)


def _values(x, s, mode):
    """What an activation or its checkpoint stands for, in 32 bits."""
    v = x.float()
    if mode == "none":
        return v
    if mode == "tensor":
        return v * s
    if mode == "mx128":
        s = 1.0 / _power(s.to(torch.int32))
    return (_blocks(v) * s[..., None]).flatten(-2)


def _plain(st):
    case = st["case"]
    op, mode, k = case["op"], case["mode"], case["k"]
    if op == "layernorm":
        h = st["X"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        d = h - h.mean(dim=-1, keepdim=True)
        y = d * torch.rsqrt((d * d).mean(dim=-1, keepdim=True) + EPS[op]) * st["weight"].float()
        if st["bias"] is not None:
            y = y + st["bias"].float()
        if mode == "none":
            out = [y.to(torch.bfloat16)]
        else:
            q, s = _quantize(y, mode, st["scale"])
            out = [q.to(torch.float8_e4m3fn)]
            if mode != "tensor":
                out.append(s.view(torch.float8_e8m0fnu) if mode == "mx128" else s)
        return out if st["residual"] is None else out + [h.to(st["X"].dtype)]
    x, dy = _values(st["X"], st["sX"], mode), st["dY"].float()
    if op == "wgrad":
        dtype = TYPES[case["out"]]
        if "m" in case:
            return [torch.mm(dy.t(), x).to(dtype)]
        if case["gather"]:
            x = x[st["rows"]]
        parts = zip(torch.split(dy, st["counts"]), torch.split(x, st["counts"]))
        return [torch.stack([torch.mm(d.t(), v).to(dtype) for d, v in parts])]
    dtype = st["dY"].dtype
    if op == "swiglu_backward":
        gate, up = x.chunk(2, dim=-1)
        s = 1.0 / (1.0 + torch.exp(-gate))
        return [torch.cat([dy * up * s * (1.0 + gate * (1.0 - s)), dy * gate * s], dim=-1).to(dtype)]
    if op == "layernorm_backward":
        x = x - x.mean(dim=-1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS[op[:-9]])
    xhat = x * rstd
    g = dy * st["weight"].float()
    dx = g - xhat * (g * xhat).mean(dim=-1, keepdim=True)
    if op == "layernorm_backward":
        dx = dx - g.mean(dim=-1, keepdim=True)
    dx = dx * rstd
    if st["residual"] is not None:
        dx = dx + st["residual"].float()
    out = [dx.to(dtype), (dy * xhat).sum(dim=0)]
    return out + [dy.sum(dim=0)] if op == "layernorm_backward" else out


# ------------------------------------------------------- the library's calls

def _own(st):
    import dense_gemm_packer_amd as dgp
    case = st["case"]
    op, mode, k = case["op"], case["mode"], case["k"]
    code = {"none": dgp.SCALE_NONE, "tensor": dgp.SCALE_TENSOR, "block128": dgp.SCALE_BLOCK128, "mx128": dgp.SCALE_MX128}[mode]
    if op == "layernorm":
        got = dgp.layernorm_quantize(st["X"], st["weight"], st["bias"], code, residual=st["residual"],
                                     scale=st["scale"] if mode == "tensor" else None)
        tail = list(got[2:])
        if mode in ("none", "tensor"):
            return [got[0]] + tail
        return [got[0], got[1].view(torch.float8_e8m0fnu) if mode == "mx128" else got[1]] + tail
    if op == "wgrad":
        return [dgp.gemm_wgrad(st["dY"], st["X"], st["sX"], code, offsets=st.get("offsets"), rows=st.get("rows"),
                               out_dtype=TYPES[case["out"]])]
    if op == "swiglu_backward":
        X, s = st["X"], st["sX"]
        sg, su = (s[:, :k // 128], s[:, k // 128:]) if mode in ("block128", "mx128") else (s, s)
        return [dgp.swiglu_backward(st["dY"], X[:, :k], X[:, k:], code, gate_scales=sg, up_scales=su)]
    fn = dgp.layernorm_backward if op == "layernorm_backward" else dgp.rmsnorm_backward
    return list(fn(st["dY"], st["X"], st["weight"], code, scales=st["sX"], residual_grad=st["residual"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ 64 bits

def _pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _to_e4m3(v):
    """v rounded to nearest even on the e4m3 grid, saturating."""
    step = _pow2(torch.clamp(torch.frexp(v)[1].to(torch.int64) - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _wide(x, s, mode):
    """What an activation or its checkpoint stands for, in 64 bits."""
    v = x.to(torch.float64)
    if mode == "none":
        return v
    if mode == "mx128":
        s = _pow2(s.to(torch.int64) - 127)
    s = s.to(torch.float64)
    return v * (s if mode == "tensor" else s.repeat_interleave(128, 1))


def exact(case, seed):
    st = prepare(case, seed)
    op, mode, k = case["op"], case["mode"], case["k"]
    if op == "layernorm":
        h = st["X"].double() if st["residual"] is None else st["X"].double() + st["residual"].double()
        mu = h.sum(dim=1, keepdim=True) / k
        y = (h - mu) / torch.sqrt((h - mu).pow(2).sum(dim=1, keepdim=True) / k + 1e-5) * st["weight"].double()
        if st["bias"] is not None:
            y = y + st["bias"].double()
        tail = [] if st["residual"] is None else [h]
        if mode == "none":
            return [y] + tail
        if mode == "tensor":
            return [_to_e4m3(y / st["scale"].double())] + tail
        big = y.abs().reshape(case["m"], k // 128, 128).max(dim=2)[0]
        if mode == "block128":
            s = torch.clamp(big / 448, min=2.0 ** -126)
        else:
            e = torch.frexp(big)[1].to(torch.int64) - 9
            e = e + (big > 448 * _pow2(torch.clamp(e, min=-200))).to(torch.int64)
            s = _pow2(torch.where(big > 0, torch.clamp(e, min=-127), -127))
        return [_to_e4m3(y / s.repeat_interleave(128, 1)), s] + tail
    x, dy = _wide(st["X"], st["sX"], mode), st["dY"].double()
    if op == "wgrad":
        if "m" in case:
            return [dy.t().contiguous() @ x]
        off = st["offsets"].tolist()
        out = torch.zeros(case["e"], case["n"], k, dtype=torch.float64, device=DEV)
        for e in range(case["e"]):
            lo, hi = off[e], off[e + 1]
            mine = x[st["rows"][lo:hi].long()] if case["gather"] else x[lo:hi]
            out[e] = dy[lo:hi].t().contiguous() @ mine
        return [out]
    if op == "swiglu_backward":
        gate, up = x[:, :k], x[:, k:]
        s = torch.sigmoid(gate)
        return [torch.cat([dy * up * (s + gate * s * torch.sigmoid(-gate)), dy * gate * s], dim=1)]
    g = dy * st["weight"].double()
    if op == "layernorm_backward":
        x = x - x.sum(dim=1, keepdim=True) / k
        inv = 1 / torch.sqrt(x.pow(2).sum(dim=1, keepdim=True) / k + 1e-5)
        g = g - g.sum(dim=1, keepdim=True) / k
    else:
        inv = 1 / torch.sqrt(x.pow(2).sum(dim=1, keepdim=True) / k + 1e-6)
    # d(x * inv)/dx applied to g: inv * g - x * inv^3 * <x, g> / k
    dx = inv * g - x * inv.pow(3) * ((x * g).sum(dim=1, keepdim=True) / k)
    if st["residual"] is not None:
        dx = dx + st["residual"].double()
    out = [dx, (dy * (x * inv)).sum(dim=0)]
    return out + [dy.sum(dim=0)] if op == "layernorm_backward" else out
