"""Operators of 8-bit training and decoding of a linear layer, as cases to be timed and compared.

  quantize   e4m3 codes with one fp32 scale per block of 128: blocks of 1 x 128 along the
             contraction (activations, gradients) or 128 x 128 (weights), of x, of its transpose,
             or of both in one pass
  product    C = A B^T of two such operands, with an optional column bias or source matrix
  norm       layer norm's forward pass
  norm_grad  its backward pass, with the gradients of the weight and the bias
  clip       the global norm of a list of gradients, and the list scaled to a largest norm

With `own` false, run() computes them from elementary torch operations; with `own` true, by the
calls of dense_gemm_design_amd.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale: a block of zeros has it


def _up(n, m):
    return -(-n // m) * m


def _blocks(n):
    return -(-n // BLOCK)


# ---- the cases --------------------------------------------------------------------------------

def listed():
    return [
        # the input of a linear layer in training: its codes along the features for the forward
        # product, and along the tokens for the weight gradient's
        {"name": "quantize_activations", "op": "quantize", "rows": 8192, "cols": 4096,
         "dtype": "bf16", "block": "row", "sides": "both", "pow2": False},
        # fp32 master weights of the MLP's up projection after an optimiser step, for the forward
        # and the input gradient's product; scales that are powers of two
        {"name": "quantize_weight", "op": "quantize", "rows": 14336, "cols": 4096,
         "dtype": "f32", "block": "tile", "sides": "both", "pow2": True},
        # one token of one sequence through a square projection
        {"name": "product_token", "op": "product", "M": 1, "N": 4096, "K": 4096, "b": "tile",
         "pow2": False, "out": "bf16", "extra": "none"},
        # the MLP's up projection over a batch of tokens, with its bias
        {"name": "product_mlp_up", "op": "product", "M": 4096, "N": 14336, "K": 4096, "b": "tile",
         "pow2": False, "out": "bf16", "extra": "bias"},
        # a large square product with scales that are powers of two
        {"name": "product_square", "op": "product", "M": 8192, "N": 8192, "K": 8192, "b": "tile",
         "pow2": True, "out": "bf16", "extra": "none"},
        # a weight gradient over an odd count of tokens, added to the fp32 sum of earlier batches
        {"name": "product_weight_grad", "op": "product", "M": 1000, "N": 4104, "K": 8201,
         "b": "row", "pow2": False, "out": "f32", "extra": "source"},
        # the norm before a linear layer, in training
        {"name": "norm_batch", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "wtype": "f32"},
        # a few sequences' single tokens, an odd width
        {"name": "norm_tokens", "op": "norm", "rows": 5, "cols": 1111, "dtype": "f32",
         "wtype": "f32"},
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 16384, "cols": 4096,
         "dtype": "bf16", "wtype": "f32"},
        # a small model's norm in fp32, with an odd width and few rows
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 515, "cols": 1111,
         "dtype": "f32", "wtype": "f32"},
        # the gradients of a model of 0.26 G parameters: bf16 matrices, fp32 vectors
        {"name": "clip_model", "op": "clip", "layers": 24, "width": 1024, "odd": 0, "clip": True},
        # the gradients of one small block, where the launches count
        {"name": "clip_block", "op": "clip", "layers": 1, "width": 96, "odd": 3, "clip": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "norm_grad", "clip"])
    if op == "quantize":
        block = rng.choice(["row", "tile"])
        rows, cols = _log(rng, 1, 16384), _log(rng, 64, 16384)
        while rows * cols > 14336 * 4096:
            rows = _log(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"]),
                "block": block, "sides": rng.choice(["one", "other", "both"]),
                "pow2": rng.random() < 0.5}
    if op == "product":
        N, K = _log(rng, 64, 16384), _log(rng, 64, 16384)
        M = _log(rng, 1, 8192)
        while M * N * K > 2 ** 37:
            M = _log(rng, 1, 8192)
        if rng.random() < 0.5:
            N, K = _up(N, 64), _up(K, 64)
        return {"op": op, "M": M, "N": N, "K": K, "b": rng.choice(["tile", "tile", "row"]),
                "pow2": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"]),
                "extra": rng.choice(["none", "bias", "source"])}
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 48, 20000)
        rows = _log(rng, 1, 16384)
        while rows * cols > 2 ** 26:
            rows = _log(rng, 1, 16384)
        if rng.random() < 0.5:
            cols = _up(cols, 64)
        dtype = rng.choice(["bf16", "f32"])
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype,
                "wtype": rng.choice(["f32", dtype])}
    return {"op": op, "layers": rng.randint(1, 24), "width": _log(rng, 32, 1200),
            "odd": rng.choice([0, rng.randint(1, 64)]), "clip": rng.random() < 0.7}


def _sizes(case):
    """The gradients' sizes: per layer two square and two four times as long matrices (bf16) and
    the vectors of two norms and the biases (fp32)."""
    w, odd = case["width"], case["odd"]
    layer = [("bf16", (w + odd) * w), ("f32", w + odd), ("bf16", w * (4 * w + odd)),
             ("f32", 4 * w + odd), ("bf16", 4 * w * w), ("f32", w), ("bf16", w * w), ("f32", w)]
    return layer * case["layers"] + [("bf16", 8 * w * w + odd)]


# ---- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _activations(g, rows, cols):
    """Values of a trained layer's input: unit normals, a few features many times larger."""
    x = _randn(g, rows, cols)
    loud = torch.rand(cols, generator=g, device=DEVICE) < 0.01
    return x * torch.where(loud, 12.0, 1.0)


def _operand(g, rows, K, block, pow2, spread):
    """e4m3 codes (rows, K up to a multiple of 16, zeros behind K) and scales of an operand."""
    x = (_activations(g, rows, K) * spread).to(torch.bfloat16)
    codes, scales = _quantize(x, block, pow2)
    held = torch.zeros(rows, _up(K, 16), dtype=torch.uint8, device=DEVICE)
    held[:, :K] = codes.view(torch.uint8)
    return held, scales.t().contiguous().t()  # the scales of one block column next to each other


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        x = _activations(g, case["rows"], case["cols"])
        if case["block"] == "tile":
            x = x * 0.02
        s["x"] = x.to(TYPES[case["dtype"]])
    elif op == "product":
        s["a"], s["sa"] = _operand(g, case["M"], case["K"], "row", case["pow2"], 1.0)
        s["b"], s["sb"] = _operand(g, case["N"], case["K"], case["b"], case["pow2"],
                                   0.02 if case["b"] == "tile" else 1.0)
        s["bias"] = _randn(g, case["N"]) if case["extra"] == "bias" else None
        s["source"] = _randn(g, case["M"], case["N"]) * 3 if case["extra"] == "source" else None
    elif op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        x = _activations(g, rows, cols) + 0.5
        s["x"] = x.to(TYPES[case["dtype"]])
        s["w"] = (1 + 0.1 * _randn(g, cols)).to(TYPES[case["wtype"]])
        s["b"] = (0.1 * _randn(g, cols)).to(TYPES[case["wtype"]])
        if op == "norm_grad":
            s["dy"] = (_randn(g, rows, cols) * 1e-2).to(TYPES[case["dtype"]])
            _, s["mean"], s["rstd"] = _norm(s["x"], s["w"], s["b"], 1e-5)
    else:
        sizes = _sizes(case)
        total = {t: sum(n for u, n in sizes if u == t) for t in TYPES}
        flat = {t: (_randn(g, total[t]) * 0.01).to(TYPES[t]) for t in TYPES}
        into = {t: torch.empty_like(flat[t]) for t in TYPES}
        at = {t: 0 for t in TYPES}
        s["grads"], s["into"], s["flat"] = [], [], [into["bf16"], into["f32"]]
        for t, n in sizes:
            s["grads"].append(flat[t][at[t]:at[t] + n])
            s["into"].append(into[t][at[t]:at[t] + n])
            at[t] += n
    return s


# ---- plain forms ------------------------------------------------------------------------------

def _two_to(e):
    """2^e as float64 from its bits, for whole e (a library's power may be off by a rounding)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_e4m3(v):
    """float64 values to the nearest e4m3 value, ties to even, at most 448 in size.  In 64 bits:
    a quotient of two floats next to a border must not be rounded onto it first."""
    _, e = torch.frexp(v)
    step = _two_to(torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _scale(amax, pow2):
    """The fp32 scale of blocks whose largest size is amax: amax / 448, or the next power of two
    that is not below it; never under 2^-126; NaN where amax is infinite or NaN."""
    if pow2:
        m, e = torch.frexp(amax.double() / E4M3_MAX)
        e = torch.where(m == 0.5, e - 1, e)
        s = _two_to(torch.clamp(e, min=-126)).float()
    else:
        s = torch.clamp((amax.double() / E4M3_MAX).float(), min=TINY)
    s = torch.where(amax == 0, torch.full_like(s, TINY), s)
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))


def _quantize(x, block, pow2):
    """e4m3 codes (rows, cols) and fp32 scales (rows or rows / 128, cols / 128), rounded up."""
    rows, cols = x.shape
    br = BLOCK if block == "tile" else 1
    pad = torch.zeros(_up(rows, br), _up(cols, BLOCK), dtype=torch.float32, device=x.device)
    pad[:rows, :cols] = x.float()
    blocked = pad.view(pad.shape[0] // br, br, pad.shape[1] // BLOCK, BLOCK)
    scales = _scale(blocked.abs().amax(dim=(1, 3)), pow2)
    q = _round_e4m3(blocked.double() / scales[:, None, :, None].double())
    codes = q.float().to(torch.float8_e4m3fn).view(pad.shape)[:rows, :cols]
    return codes, scales


def _spread(codes, scales, K):
    """The fp32 values that an operand's codes and scales stand for, without the zeros behind K."""
    v = codes.view(torch.float8_e4m3fn).float()[:, :K]
    rows = v.shape[0]
    s = scales if scales.shape[0] == rows and (rows > 1) else scales.repeat_interleave(BLOCK, 0)
    return v * s[:rows].repeat_interleave(BLOCK, 1)[:, :K]


def _product(s):
    case = s["case"]
    c = torch.matmul(_spread(s["a"], s["sa"], case["K"]), _spread(s["b"], s["sb"], case["K"]).t())
    if s["bias"] is not None:
        c = c + s["bias"]
    if s["source"] is not None:
        c = c + s["source"]
    return c.to(TYPES[case["out"]])


def _norm(x, w, b, eps):
    f = x.float()
    mean = f.mean(dim=1, keepdim=True)
    d = f - mean
    rstd = torch.rsqrt((d * d).mean(dim=1, keepdim=True) + eps)
    return (d * rstd * w.float() + b.float()).to(x.dtype), mean[:, 0], rstd[:, 0]


def _norm_grad(dy, x, w, mean, rstd):
    g = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    gw = g * w.float()
    dx = rstd[:, None] * (gw - gw.mean(dim=1, keepdim=True)
                          - xhat * (gw * xhat).mean(dim=1, keepdim=True))
    return dx.to(x.dtype), (g * xhat).sum(dim=0).to(w.dtype), g.sum(dim=0).to(w.dtype)


def _clip(s):
    total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
    norm = total.sqrt().float()
    if not s["case"]["clip"]:
        return [norm]
    c = torch.clamp(1.0 / (norm + 1e-6), max=1.0)
    [o.copy_(g.float() * c) for o, g in zip(s["into"], s["grads"])]
    return [norm, *s["flat"]]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import dense_gemm_design_amd as dg
    if op == "quantize":
        if own:
            side = {"one": False, "other": True, "both": "both"}[case["sides"]]
            q = dg.block_quantize(s["x"], case["block"], transposed=side, pow2=case["pow2"])
            q = q if isinstance(q, tuple) else (q,)
            return [t for o in q for t in (o.values, o.scales)]
        sides = {"one": [s["x"]], "other": [s["x"].t()], "both": [s["x"], s["x"].t()]}
        return [t for x in sides[case["sides"]] for t in _quantize(x, case["block"], case["pow2"])]
    if op == "product":
        if own:
            a = dg.BlockScaled(s["a"], s["sa"], case["K"], "row", case["pow2"])
            b = dg.BlockScaled(s["b"], s["sb"], case["K"], case["b"], case["pow2"])
            return dg.block_gemm(a, b, out_dtype=case["out"], bias_col=s["bias"],
                                 source=s["source"])
        return _product(s)
    if op == "norm":
        if own:
            return list(dg.layer_norm(s["x"], s["w"], s["b"], eps=1e-5))
        return list(_norm(s["x"], s["w"], s["b"], 1e-5))
    if op == "norm_grad":
        if own:
            return list(dg.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"]))
        return list(_norm_grad(s["dy"], s["x"], s["w"], s["mean"], s["rstd"]))
    if own:
        if not case["clip"]:
            return [dg.grad_norm(s["grads"])]
        return [dg.clip_grad_norm(s["grads"], 1.0, out=s["into"]), *s["flat"]]
    return _clip(s)


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c, n = case["rows"], case["cols"], BYTES[case["dtype"]]
        sides = 2 if case["sides"] == "both" else 1
        tile = case["block"] == "tile"
        scales = (_blocks(r) * _blocks(c) * sides if tile else
                  (case["sides"] != "other") * r * _blocks(c)
                  + (case["sides"] != "one") * c * _blocks(r))
        return {"bytes": r * c * (n + sides) + 4 * scales, "flops": r * c * (1 + sides)}
    if op == "product":
        M, N, K, kb = case["M"], case["N"], case["K"], _blocks(case["K"])
        b = (M + N) * K + 4 * kb * (M + (_blocks(N) if case["b"] == "tile" else N))
        b += M * N * BYTES[case["out"]]
        b += {"none": 0, "bias": 4 * N, "source": 4 * M * N}[case["extra"]]
        return {"bytes": b, "flops": 2 * M * N * K}
    if op in ("norm", "norm_grad"):
        r, c, n, w = case["rows"], case["cols"], BYTES[case["dtype"]], BYTES[case["wtype"]]
        if op == "norm":
            return {"bytes": 2 * r * c * n + 2 * c * w + 8 * r, "flops": 8 * r * c}
        return {"bytes": 3 * r * c * n + 3 * c * w + 8 * r, "flops": 14 * r * c}
    n = sum(BYTES[t] * k for t, k in _sizes(case))
    count = sum(k for _, k in _sizes(case))
    return {"bytes": n * (2 if case["clip"] else 1) + 4,
            "flops": count * (3 if case["clip"] else 2)}


# ---- the definitions in 64 bits, apart from the plain forms -----------------------------------

def _e4m3_table():
    """All non-negative finite e4m3 values in order: code i is the i-th."""
    v = [i / 8 * 2.0 ** -6 for i in range(8)]
    return v + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest_e4m3(v):
    """By search among the midpoints of neighbouring values; a tie takes the even code."""
    table = torch.tensor(_e4m3_table(), dtype=torch.float64, device=v.device)
    mids = (table[1:] + table[:-1]) / 2
    size = v.abs().contiguous()
    low = torch.searchsorted(mids, size, right=False)   # midpoints below size
    high = torch.searchsorted(mids, size, right=True)   # midpoints at or below size
    code = torch.where(low % 2 == 0, low, high)         # on a midpoint low and high differ by one
    code = torch.where(low == high, low, code)
    near = table[code.clamp(max=126)]
    return torch.where(torch.isnan(v), v, torch.where(v < 0, -near, near))


def _exact_quantize(x, block, pow2):
    rows, cols = x.shape
    br = BLOCK if block == "tile" else 1
    values = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    scales = torch.empty(-(-rows // br), _blocks(cols), dtype=torch.float64, device=x.device)
    for j in range(_blocks(cols)):
        strip = x[:, j * BLOCK:(j + 1) * BLOCK].double()
        top = strip.abs().amax(dim=1)
        if br > 1:
            top = torch.cat([top, top.new_zeros(_up(rows, br) - rows)]).view(-1, br).amax(dim=1)
        if pow2:
            s = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX))).float().double()
            s = torch.where(s / 2 * E4M3_MAX >= top, s / 2, s)   # log2 may be off by a rounding
            s = torch.where(s * E4M3_MAX < top, s * 2, s)
        else:
            s = (top / E4M3_MAX).float().double()   # the scale is an fp32 number by definition
        s = s.clamp(min=TINY)
        scales[:, j] = s
        values[:, j * BLOCK:(j + 1) * BLOCK] = _nearest_e4m3(
            strip / s.repeat_interleave(br)[:rows, None])
    return values, scales


def _exact_values(codes, scales, block, K):
    table = torch.tensor(_e4m3_table() + [float("nan")], dtype=torch.float64, device=codes.device)
    table = torch.cat([table, -table])
    v = table[codes.long()]
    for j in range(_blocks(K)):
        s = scales[:, j].double()
        s = s.repeat_interleave(BLOCK)[:v.shape[0]] if block == "tile" else s
        v[:, j * BLOCK:(j + 1) * BLOCK] *= s[:, None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        sides = {"one": [s["x"]], "other": [s["x"].t()], "both": [s["x"], s["x"].t()]}
        return [t for x in sides[case["sides"]]
                for t in _exact_quantize(x, case["block"], case["pow2"])]
    if op == "product":
        a = _exact_values(s["a"], s["sa"], "row", case["K"])
        b = _exact_values(s["b"], s["sb"], case["b"], case["K"])
        c = torch.mm(a, b.t().contiguous())
        for extra in (s["bias"], s["source"]):
            if extra is not None:
                c += extra.double()
        return c
    if op in ("norm", "norm_grad"):
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        n = x.shape[1]
        if op == "norm":
            mean = x.sum(1) / n
            var = ((x - mean[:, None]) ** 2).sum(1) / n
            rstd = (var + 1e-5) ** -0.5
            return [(x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd]
        dy, mean, rstd = s["dy"].double(), s["mean"].double(), s["rstd"].double()
        xhat = (x - mean[:, None]) * rstd[:, None]
        inner = dy * w - (dy * w).sum(1)[:, None] / n - xhat * ((dy * w * xhat).sum(1) / n)[:, None]
        return [inner * rstd[:, None], (dy * xhat).sum(0), dy.sum(0)]
    norm = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in s["grads"]))
    if not case["clip"]:
        return [torch.tensor(norm, dtype=torch.float64)]
    c = min(1.0, 1.0 / (norm + 1e-6))
    parts = {t: [g.double() * c for g in s["grads"] if g.dtype == TYPES[t]] for t in TYPES}
    return [torch.tensor(norm, dtype=torch.float64), torch.cat(parts["bf16"]),
            torch.cat(parts["f32"])]
