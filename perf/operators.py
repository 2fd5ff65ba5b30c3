"""Cases of the block-scaled 8-bit linear layer: RMS norm with the residual's addition and an 8-bit
output, its gradient, the block quantiser, and the 8-bit matrix product with a scale for each block of 128.

8-bit values are e4m3; scales are powers of two held in one byte (E8M0: the byte minus 127 is the exponent).
The plain forms below are elementary torch operations in 32 bits; with `own` set, run() makes the calls that
a user makes of the package.
"""
import math

import torch

own = False

BLOCK = 128


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one sample's token through the norm of a serving step: latency only
        {"name": "norm one row", "op": "norm", "rows": 1, "D": 1536, "dtype": "bf16", "resid": True, "plain": False},
        # a training batch of 512 samples x 32 tokens: residual stream, 8-bit rows and what the gradient needs
        {"name": "norm batch", "op": "norm", "rows": 16384, "D": 1536, "dtype": "bf16", "resid": True, "plain": True},
        # wide fp32 stream whose last block of 128 is ragged and whose rows are odd in number
        {"name": "norm wide f32", "op": "norm", "rows": 4099, "D": 7184, "dtype": "f32", "resid": False, "plain": False},
        # the gradient of the batch above
        {"name": "norm grad batch", "op": "norm_grad", "rows": 16384, "D": 1536, "dtype": "bf16", "dsum": True},
        # few wide rows: the column sums dominate the latency
        {"name": "norm grad few rows", "op": "norm_grad", "rows": 37, "D": 5120, "dtype": "f32", "dsum": False},
        # all first-projection weights of a block, once per optimizer step: both orientations, 128 x 128 blocks
        {"name": "quantize weights", "op": "quantize", "G": 32, "rows": 6144, "cols": 1536, "block_rows": 128,
         "dtype": "bf16", "tokens": False, "both": True},
        # activations [samples, tokens, width]: rows for the forward product, columns for the weight gradient
        {"name": "quantize tokens", "op": "quantize", "G": 16, "rows": 509, "cols": 768, "block_rows": 1,
         "dtype": "bf16", "tokens": True, "both": True},
        # one row through one projection: the smallest product
        {"name": "product one row", "op": "product", "G": 1, "M": 1, "N": 1536, "K": 1536, "block_rows": 128,
         "out": "bf16", "act": "none", "bias": False, "resid": False},
        # a serving step of four samples: every token's weights are streamed once
        {"name": "product four samples", "op": "product", "G": 32, "M": 4, "N": 6144, "K": 1536, "block_rows": 128,
         "out": "e4m3", "act": "tanh", "bias": True, "resid": False},
        # first projection of the batch of 512: bias, GELU, 8-bit hidden for the second projection
        {"name": "product batch", "op": "product", "G": 32, "M": 512, "N": 6144, "K": 1536, "block_rows": 128,
         "out": "e4m3", "act": "tanh", "bias": True, "resid": False},
        # odd sizes: ragged tiles in every direction, residual added
        {"name": "product ragged", "op": "product", "G": 5, "M": 333, "N": 1104, "K": 2064, "block_rows": 128,
         "out": "bf16", "act": "none", "bias": True, "resid": True},
        # weight gradient: both operands have a scale for each row's 128 samples, fp32 result
        {"name": "product weight grad", "op": "product", "G": 32, "M": 6144, "N": 1536, "K": 512, "block_rows": 1,
         "out": "f32", "act": "none", "bias": False, "resid": False},
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of `step` from lo to hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "quantize", "quantize", "product", "product", "product"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        D = _between(rng, 64, 8192, 16)
        rows = _between(rng, 1, min(32768, 25_000_000 // D))
        if op == "norm":
            return {"op": op, "rows": rows, "D": D, "dtype": dtype, "resid": rng.random() < 0.6,
                    "plain": rng.random() < 0.5}
        return {"op": op, "rows": rows, "D": D, "dtype": dtype, "dsum": rng.random() < 0.6}
    if op == "quantize":
        G, cols = _between(rng, 1, 32), _between(rng, 64, 6144, 16)
        rows = _between(rng, 1, min(8192, 200_000_000 // (G * cols)))
        return {"op": op, "G": G, "rows": rows, "cols": cols, "block_rows": rng.choice([1, 128]), "dtype": dtype,
                "tokens": rng.random() < 0.5, "both": rng.random() < 0.6}
    G = _between(rng, 1, 32)
    N, K = _between(rng, 64, 6144, 16), _between(rng, 64, 6144, 16)
    M = _between(rng, 1, max(1, min(6144, 150_000_000_000 // (G * N * K))))
    while G * N * max(M, K) > 320_000_000:
        G = max(1, G // 2)
    out = rng.choice(["bf16", "bf16", "f32", "e4m3"])
    return {"op": op, "G": G, "M": M, "N": N, "K": K, "block_rows": rng.choice([1, 128, 128]), "out": out,
            "act": rng.choice(["none", "none", "tanh", "erf", "relu"]), "bias": rng.random() < 0.5,
            "resid": out != "e4m3" and rng.random() < 0.4}


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-5


def _blocks(n):
    return -(-n // BLOCK)


def _up(n, k):
    return -(-n // k) * k


def work(case):
    c = case
    if c["op"] == "norm":
        e, n = _BYTES[c["dtype"]], c["rows"] * c["D"]
        per = e * (1 + 2 * c["resid"] + c["plain"]) + 1
        return {"bytes": n * per + c["rows"] * (_blocks(c["D"]) + 4) + 4 * c["D"], "flops": 6 * n}
    if c["op"] == "norm_grad":
        e, n = _BYTES[c["dtype"]], c["rows"] * c["D"]
        return {"bytes": n * e * (3 + c["dsum"]) + 4 * c["rows"] + 8 * c["D"], "flops": 10 * n}
    if c["op"] == "quantize":
        n = c["G"] * c["rows"] * c["cols"]
        return {"bytes": n * (_BYTES[c["dtype"]] + 1 + c["both"]), "flops": 2 * n}
    G, M, N, K = c["G"], c["M"], c["N"], c["K"]
    inputs = G * (M * K + N * K + M * _blocks(K) + -(-N // c["block_rows"]) * _blocks(K) + 4 * N * c["bias"])
    return {"bytes": inputs + G * M * N * _BYTES[c["out"]] * (1 + c["resid"]), "flops": 2 * G * M * N * K}


# ---------------------------------------------------------------------------- 8-bit blocks, plain
def _exponent(amax):
    """Smallest e in [-127, 127] with amax <= 448 * 2^e; 0 for a zero block."""
    m, e = torch.frexp(amax)                      # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _amax(x, block_rows):
    """Largest magnitude of each block_rows x 128 block of x [..., rows, cols]."""
    rows, cols = x.shape[-2:]
    a = torch.nn.functional.pad(x.abs(), (0, _up(cols, BLOCK) - cols, 0, _up(rows, block_rows) - rows))
    return a.unflatten(-1, (-1, BLOCK)).amax(-1).unflatten(-2, (-1, block_rows)).amax(-2)


def _spread(e, rows, cols, block_rows):
    return e.repeat_interleave(block_rows, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _quantize(x, block_rows):
    """e4m3 codes and E8M0 scale bytes of x [..., rows, cols]."""
    rows, cols = x.shape[-2:]
    e = _exponent(_amax(x, block_rows))
    q = torch.ldexp(x, -_spread(e, rows, cols, block_rows)).float().to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _values(q, scale, block_rows, dtype=torch.float32):
    e = scale.to(torch.int32) - 127
    return torch.ldexp(q.to(dtype), _spread(e, q.shape[-2], q.shape[-1], block_rows))


def _activation(v, act):
    if act == "tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "erf":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v.clamp(min=0) if act == "relu" else v


# ---------------------------------------------------------------------------- inputs
def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _stream(g, rows, D, dtype):
    """A residual stream: rows of different size, a few channels much larger than the others."""
    size = torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    channel = torch.exp(0.7 * torch.randn((1, D), generator=g, device="cuda"))
    return (torch.randn((rows, D), generator=g, device="cuda") * size * channel).to(dtype)


def _padded(shape):
    """e4m3 buffer [..., n] whose rows start on 16-byte boundaries."""
    return torch.zeros(shape[:-1] + (_up(shape[-1], 16),), dtype=torch.float8_e4m3fn, device="cuda")[..., :shape[-1]]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("norm", "norm_grad"):
        rows, D, dt = c["rows"], c["D"], _TYPES[c["dtype"]]
        s["gamma"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s["x"] = _stream(g, rows, D, dt)
        if c["op"] == "norm":
            s["r"] = _normal(g, (rows, D), dt) if c["resid"] else None
            s["sum"] = torch.empty_like(s["x"]) if c["resid"] else None
            s["y"] = torch.empty_like(s["x"]) if c["plain"] else None
            s["yq"] = torch.empty((rows, D), dtype=torch.float8_e4m3fn, device="cuda")
            s["ys"] = torch.empty((rows, _blocks(D)), dtype=torch.uint8, device="cuda")
            s["rstd"] = torch.empty(rows, device="cuda")
        else:
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(-1) + EPS).float()
            s["dy"] = _normal(g, (rows, D), dt, 0.1)
            s["dsum"] = _normal(g, (rows, D), dt, 0.1) if c["dsum"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(D, device="cuda")
            s["ws"] = torch.empty(1024 * D, device="cuda")   # the column sums' partials
        return s
    if c["op"] == "quantize":
        G, rows, cols, dt, br = c["G"], c["rows"], c["cols"], _TYPES[c["dtype"]], c["block_rows"]
        if c["tokens"]:   # [rows, G, cols] in memory, as activations [B, T, D]
            s["x"] = _normal(g, (rows, G, cols), dt).transpose(0, 1)
        else:
            s["x"] = _normal(g, (G, rows, cols), dt, (2 / (rows + cols)) ** 0.5)
        s["q"] = torch.empty((G, rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.empty((G, -(-rows // br), _blocks(cols)), dtype=torch.uint8, device="cuda")
        s["qt"] = _padded((G, cols, rows)) if c["both"] else None
        s["st"] = torch.empty((G, -(-cols // br), _blocks(rows)), dtype=torch.uint8, device="cuda") if c["both"] else None
        return s
    G, M, N, K, br = c["G"], c["M"], c["N"], c["K"], c["block_rows"]
    s["a"], s["as"], s["w"] = _padded((G, M, K)), torch.empty((G, M, _blocks(K)), dtype=torch.uint8, device="cuda"), _padded((G, N, K))
    s["ws"] = torch.empty((G, -(-N // br), _blocks(K)), dtype=torch.uint8, device="cuda")
    for i in range(G):
        a, s["as"][i] = _quantize(_normal(g, (M, K), torch.bfloat16).float(), 1)
        w, s["ws"][i] = _quantize(_normal(g, (N, K), torch.bfloat16, (2 / (N + K)) ** 0.5).float(), br)
        s["a"][i], s["w"][i] = a, w
    s["bias"] = _normal(g, (G, N), torch.float32, 0.1) if c["bias"] else None
    s["resid"] = _normal(g, (G, M, N), _TYPES[c["out"]]) if c["resid"] else None
    s["out"] = torch.empty((G, M, N), dtype=_TYPES[c["out"]], device="cuda")
    s["os"] = torch.empty((G, M, _blocks(N)), dtype=torch.uint8, device="cuda") if c["out"] == "e4m3" else None
    return s


# ---------------------------------------------------------------------------- one pass
def _scales(s):
    return None if s is None else s.view(torch.float8_e8m0fnu)


def _norm(s, real):
    """The norm's outputs with its arithmetic in type `real`."""
    x, c = s["x"], s["case"]
    if s["r"] is not None:
        x = (x.float() + s["r"].float()).to(x.dtype)      # the stream as it is stored
    v = x.to(real)
    rstd = torch.rsqrt(v.square().mean(-1) + EPS)
    y = v * rstd[:, None] * s["gamma"].to(real)
    q, sc = _quantize(y, 1)
    keep = torch.float64 if real is torch.float64 else x.dtype
    return {"sum": x if s["r"] is not None else None, "y": y.to(keep) if c["plain"] else None, "q": q, "s": _scales(sc),
            "rstd": rstd}


def _norm_grad(s, real):
    x, dy, rstd = s["x"].to(real), s["dy"].to(real), s["rstd"].to(real)[:, None]
    a = dy * s["gamma"].to(real)
    dx = rstd * (a - x * rstd.square() * (a * x).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].to(real)
    return {"dx": dx if real is torch.float64 else dx.to(s["x"].dtype), "dgamma": (dy * x * rstd).sum(0)}


def _quantize_both(s):
    br, x = s["case"]["block_rows"], s["x"].float()
    q, sc = _quantize(x, br)
    if s["qt"] is None:
        return {"q": q, "s": _scales(sc)}
    qt, st = _quantize(x.transpose(-2, -1), br)
    return {"q": q, "s": _scales(sc), "qt": qt, "st": _scales(st)}


def _product(s, real):
    c = s["case"]
    a = _values(s["a"], s["as"], 1, real)
    w = _values(s["w"], s["ws"], c["block_rows"], real)
    v = torch.bmm(a, w.transpose(1, 2))
    if s["bias"] is not None:
        v = v + s["bias"].to(real)[:, None]
    v = _activation(v, c["act"])
    if s["resid"] is not None:
        v = v + s["resid"].to(real)
    if c["out"] == "e4m3":
        q, sc = _quantize(v, 1)
        return {"out": q, "s": _scales(sc)}
    return {"out": v if real is torch.float64 else v.to(_TYPES[c["out"]])}


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from token_mixing_feature_b200 import rankmixer as rm
        if op == "norm":
            rm.rm_rmsnorm_forward(s["x"], s["r"], s["gamma"], s["sum"], s["y"], s["yq"], s["ys"], s["rstd"], EPS)
            return {"sum": s["sum"], "y": s["y"], "q": s["yq"], "s": _scales(s["ys"]), "rstd": s["rstd"]}
        if op == "norm_grad":
            rm.rm_rmsnorm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], s["dsum"], s["dx"], s["dgamma"], s["ws"])
            return {"dx": s["dx"], "dgamma": s["dgamma"]}
        if op == "quantize":
            rm.rm_quantize_fp8_block(s["x"], s["q"], s["s"], s["qt"], s["st"], s["case"]["block_rows"])
            out = {"q": s["q"], "s": _scales(s["s"])}
            return out if s["qt"] is None else {**out, "qt": s["qt"], "st": _scales(s["st"])}
        rm.rm_matmul_fp8_block(s["a"], s["as"], s["w"], s["ws"], s["out"], s["os"], s["bias"], s["case"]["act"],
                               s["resid"], s["case"]["block_rows"])
        return {"out": s["out"]} if s["os"] is None else {"out": s["out"], "s": _scales(s["os"])}
    if op == "norm":
        return _norm(s, torch.float32)
    if op == "norm_grad":
        return _norm_grad(s, torch.float32)
    return _quantize_both(s) if op == "quantize" else _product(s, torch.float32)


# ---------------------------------------------------------------------------- 64 bits
def _code(v):
    """Nearest e4m3 value of v (64 bits, |v| <= 448), ties to even, from the format's definition."""
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -6))
    step = torch.ldexp(torch.ones_like(v), e - 4)     # 3 bits behind the leading one; 2^-9 below 2^-6
    return torch.round(v / step) * step


def _exact_blocks(v):
    """Codes and scales (as the values they stand for) of rows of 128 of v [..., n], in 64 bits."""
    n = v.shape[-1]
    amax = torch.nn.functional.pad(v, (0, _up(n, BLOCK) - n)).unflatten(-1, (-1, BLOCK)).abs().amax(-1)
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448))
    e = torch.where(torch.ldexp(torch.full_like(e, 448), e - 1) >= amax, e - 1, e)      # log2 next to a border
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    scale = torch.exp2(e)
    return _code(v / scale.repeat_interleave(BLOCK, -1)[..., :n]), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        if s["r"] is not None:
            x = (x + s["r"].double()).to(s["x"].dtype).double()
        rstd = 1 / torch.sqrt((x * x).sum(1) / case["D"] + EPS)
        y = torch.einsum("rd,r,d->rd", x, rstd, s["gamma"].double())
        q, scale = _exact_blocks(y)
        return {"sum": x if s["r"] is not None else None, "y": y if case["plain"] else None, "q": q, "s": scale, "rstd": rstd}
    if op == "norm_grad":
        x, dy, r, gam = s["x"].double(), s["dy"].double(), s["rstd"].double(), s["gamma"].double()
        dot = torch.einsum("rd,rd,d->r", x, dy, gam)
        dx = torch.einsum("rd,d,r->rd", dy, gam, r) - torch.einsum("rd,r->rd", x, dot * r ** 3 / case["D"])
        if s["dsum"] is not None:
            dx += s["dsum"].double()
        return {"dx": dx, "dgamma": torch.einsum("rd,rd,r->d", x, dy, r)}
    if op == "quantize":
        x = s["x"].double()
        out = {}
        for key, v in (("", x), ("t", x.transpose(1, 2))) if s["qt"] is not None else (("", x),):
            G, rows, cols = v.shape
            if case["block_rows"] == 1:
                out["q" + key], out["s" + key] = _exact_blocks(v)
                continue
            p = torch.nn.functional.pad(v, (0, _up(cols, BLOCK) - cols, 0, _up(rows, BLOCK) - rows))
            p = p.reshape(G, _blocks(rows), BLOCK, _blocks(cols), BLOCK).transpose(2, 3).flatten(3)   # one row a block
            p = p.abs().amax(-1, keepdim=True)
            scale = _exact_blocks(p)[1]
            wide = scale[..., 0].repeat_interleave(BLOCK, 1)[:, :rows].repeat_interleave(BLOCK, 2)[..., :cols]
            out["q" + key], out["s" + key] = _code(v / wide), scale[..., 0]
        return out
    a = s["a"].double() * torch.exp2(s["as"].double() - 127).repeat_interleave(BLOCK, 2)[..., :case["K"]]
    w = s["w"].double() * torch.exp2(s["ws"].double() - 127).repeat_interleave(case["block_rows"], 1)[:, :case["N"]] \
        .repeat_interleave(BLOCK, 2)[..., :case["K"]]
    v = torch.einsum("gmk,gnk->gmn", a, w)
    if s["bias"] is not None:
        v += s["bias"].double()[:, None]
    if case["act"] == "tanh":
        v = v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
    elif case["act"] == "erf":
        v = v * torch.special.ndtr(v)
    elif case["act"] == "relu":
        v = torch.where(v > 0, v, torch.zeros_like(v))
    if s["resid"] is not None:
        v += s["resid"].double()
    if case["out"] == "e4m3":
        q, scale = _exact_blocks(v)
        return {"out": q, "s": scale}
    return {"out": v}
