"""Plain forms, in 64 bits, of the operators around the product, for their tests."""
import torch

U = 2.0 ** -24          # half a step of fp32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}

_POSITIVE = [i / 8 * 2.0 ** -6 for i in range(8)]
_POSITIVE += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def decode(codes):
    """float64 values of uint8 e4m3 codes."""
    t = torch.tensor(_POSITIVE + [float("nan")], dtype=torch.float64)
    return torch.cat([t, -t])[codes.cpu().long()]


def encode(v):
    """The uint8 e4m3 codes nearest to float64 values of at most 448 (1 + 2^-24), ties to the even
    code, by search; 0x7F for NaN."""
    table = torch.tensor(_POSITIVE, dtype=torch.float64)
    mids = (table[1:] + table[:-1]) / 2
    size = v.abs().contiguous()
    low, high = torch.searchsorted(mids, size), torch.searchsorted(mids, size, right=True)
    code = torch.where((low != high) & (low % 2 == 1), high, low).clamp(max=126)
    code = torch.where(torch.signbit(v), code + 128, code)
    return torch.where(torch.isnan(v), torch.full_like(code, 127), code).to(torch.uint8)


def up(n, m):
    return -(-n // m)


def quantize(x, block, pow2):
    """(codes with zeros behind each row up to a multiple of 16, float32 scales) of a CPU tensor."""
    rows, cols = x.shape
    br = 128 if block == "tile" else 1
    codes = torch.zeros(rows, up(cols, 16) * 16, dtype=torch.uint8)
    scales = torch.empty(up(rows, br), up(cols, 128), dtype=torch.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            b = x[i * br:(i + 1) * br, j * 128:(j + 1) * 128].double()
            top = float(b.abs().max()) if not bool(torch.isnan(b).any()) else float("nan")
            if top != top or top == float("inf"):
                s = float("nan")
            elif pow2:
                s = 2.0 ** -126
                while s * 448 < top:
                    s *= 2
            else:
                s = max(float(torch.tensor(top / 448.0, dtype=torch.float64).float()), 2.0 ** -126)
            scales[i, j] = s
            codes[i * br:(i + 1) * br, j * 128:j * 128 + b.shape[1]] = encode(b / s)
    return codes, scales


def spread(codes, scales, block, K):
    """float64 (rows, K) that codes and scales stand for."""
    v = decode(codes)[:, :K]
    s = scales.cpu().double().repeat_interleave(128, 1)[:, :K]
    return v * (s.repeat_interleave(128, 0)[:v.shape[0]] if block == "tile" else s)


def norm(x, w, b, eps):
    x, w = x.double(), w.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = ((d * d).mean(1) + eps) ** -0.5
    y = d * rstd[:, None] * w
    return (y + b.double() if b is not None else y), mean, rstd


def norm_grad(dy, x, w, mean, rstd):
    dy, x, w, mean, rstd = (t.double() for t in (dy, x, w, mean, rstd))
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def within(got, want, bound, what=""):
    """Every element of got within bound of want; the same ones NaN or infinite."""
    got, want, bound = got.double().cpu(), want.double().cpu(), bound.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    same = torch.equal(torch.isnan(got), torch.isnan(want))
    assert same and torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)]), what
    bad = ~odd & ((got - want).abs() > bound)
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        i = tuple(at)
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} outside, first at {at}: "
                             f"{float(got[i])} for {float(want[i])} +- {float(bound[i])}")
