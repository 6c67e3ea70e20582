"""The block-scaled product with scales near the ends of their range, on every kernel: few rows, tiles
of 128 (one or two groups of waves, K cut), of 256, and wide ones."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from test_gpu_ops import BF16, F32, dev, gen, product_bound  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# (M, N, K): few rows, with one and two blocks of rows and with K cut; 128 x 128 tiles, one and two
# groups of waves; 256 x 256 and wide tiles (bf16 C)
SHAPES = [(8, 200, 384), (30, 5000, 384), (4, 100, 5000), (300, 4400, 384), (140, 139, 5000),
          (4096, 4352, 384), (4096, 4096, 256)]
KINDS = [("row", False), ("tile", False), ("row", True), ("tile", True)]
kinds = pytest.mark.parametrize("block,pow2", KINDS,
                                ids=[f"{b}-{'pow2' if p else 'any'}" for b, p in KINDS])


def codes_of(g, rows, K):
    """Random finite codes (of all sizes), zeros behind K."""
    c = torch.randint(0, 127, (rows, R.up(K, 16) * 16), generator=g, dtype=torch.uint8)
    c |= torch.randint(0, 2, c.shape, generator=g, dtype=torch.uint8) << 7
    c[:, K:] = 0
    return c


def operand(g, dev, codes, K, block, pow2, exponents):
    """BlockScaled of codes with scales 2^e (1 to 2 times that unless pow2), e of each block of k;
    and the values."""
    rows = codes.shape[0]
    sr = R.up(rows, 128) if block == "tile" else rows
    e = torch.tensor([float(x) for x in exponents])
    m = torch.ones(sr, len(exponents)) if pow2 else 1 + torch.rand(sr, len(exponents), generator=g)
    scales = (m.double() * torch.exp2(e.double())).float()
    q = dg.BlockScaled(codes.to(dev), scales.t().contiguous().to(dev).t(), K, block, pow2)
    v = R.decode(codes).to(dev)[:, :K]
    s = scales.double().to(dev).repeat_interleave(128, 1)[:, :K]
    return q, v * (s.repeat_interleave(128, 0)[:rows] if block == "tile" else s)


def cycle(values, K):
    return [values[i % len(values)] for i in range(R.up(K, 128))]


def small_steps(blocks, dt):
    """Numbers under 2^-126 have steps of 2^-149 (bf16: 2^-133): half of one at each of three roundings a
    block, at the sums of splits and groups, and at the output's."""
    return (3 * blocks + 70) * 2.0 ** -150 + (2.0 ** -134 if dt is BF16 else 0.0)


def check(dev, a, b, av, bv, K, what):
    want = torch.mm(av, bv.t().contiguous())
    for out, dt in (("bf16", BF16), ("f32", F32)):
        got = dg.block_gemm(a, b, out_dtype=out)
        bound = product_bound(av, bv, K, want, dt, []) + small_steps(R.up(K, 128), dt)
        bad = ~((got.double() - want).abs() <= bound)
        assert not bool(bad.any()), (what, out, int(bad.sum()), bad.nonzero()[0].tolist(),
                                     float(got[bad][0]), float(want[bad][0]))


@kinds
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_blocks_that_do_not_meet_add_nothing(dev, M, N, K, block, pow2):
    """A block whose sum is zero adds zero, however large its scales; the other blocks count."""
    print(f"zero sums {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M + N + K)
    ca, cb = codes_of(g, M, K), codes_of(g, N, K)
    for j in range(0, R.up(K, 128), 3):   # every third block: no k where both have codes
        ca[:, j * 128:j * 128 + 128:2] = 0
        cb[:, j * 128 + 1:j * 128 + 128:2] = 0
    for ea, eb in ((70, 60), (118, 118), (118, 20), (20, 118)):
        a, av = operand(g, dev, ca, K, "row", pow2, cycle([ea, -10, 3], K))
        b, bv = operand(g, dev, cb, K, block, pow2, cycle([eb, 4, -9], K))
        check(dev, a, b, av, bv, K, f"2^{ea} 2^{eb}")


@kinds
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_of_any_size(dev, M, N, K, block, pow2):
    """Scales whose product is under the smallest normal number, or one of which times a block's sum is
    past the largest, where C is neither.  Sums of random codes are about 2^18 here."""
    print(f"scales of any size {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M + N + K)
    ca, cb, blocks = codes_of(g, M, K), codes_of(g, N, K), R.up(K, 128)
    # the same mantissas for every size, so that C and its bound only move by a power of two
    a, av = operand(g, dev, ca, K, "row", pow2, cycle([0, 1], K))
    b, bv = operand(g, dev, cb, K, block, pow2, cycle([1, 0], K))
    plain = torch.mm(av, bv.t().contiguous())
    bounds = {dt: product_bound(av, bv, K, plain, dt, []) for dt in (BF16, F32)}
    one_a, one_b = a.scales.clone(), b.scales.clone()
    for ea, eb in ((0, 0), (-100, -42), (-42, -100), (-125, -17), (-17, -125), (-71, -71), (-100, 110),
                   (110, -100), (-126, 118), (118, -126), (40, 45), (-126, -126)):
        a.scales.copy_(one_a * 2.0 ** ea)
        b.scales.copy_(one_b * 2.0 ** eb)
        want = plain * 2.0 ** (ea + eb)
        for out, dt in (("bf16", BF16), ("f32", F32)):
            got = dg.block_gemm(a, b, out_dtype=out)
            bound = bounds[dt] * 2.0 ** (ea + eb) + small_steps(blocks, dt)
            bad = ~((got.double() - want).abs() <= bound)
            assert not bool(bad.any()), (ea, eb, out, int(bad.sum()), bad.nonzero()[0].tolist(),
                                         float(got[bad][0]), float(want[bad][0]))


@kinds
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_blocks_of_zeros_add_nothing(dev, M, N, K, block, pow2):
    """Rows and tiles of zeros have the smallest scale, 2^-126."""
    g = gen(M + N)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    x[M // 3:M // 2 + 1] = 0
    x[:, 128:256] = 0
    w[:, 256:384] = 0
    a = dg.block_quantize(x.to(dev), "row", pow2=pow2)
    b = dg.block_quantize(w.to(dev), block, pow2=pow2)
    assert float(a.scales[M // 3, 0]) == 2.0 ** -126
    av = R.spread(a.data, a.scales, "row", K).to(dev)
    bv = R.spread(b.data, b.scales, block, K).to(dev)
    check(dev, a, b, av, bv, K, "zeros")
    assert not bool(dg.block_gemm(a, b)[M // 3:M // 2 + 1].any())


@kinds
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_of_zero_and_not_a_number(dev, M, N, K, block, pow2):
    """A NaN scale makes its row (of C) NaN and no other, its column or tile of columns likewise; a
    scale of zero (not a power of two) takes its block out."""
    g = gen(M + N)
    a, av = operand(g, dev, codes_of(g, M, K), K, "row", pow2, cycle([0, 1], K))
    b, bv = operand(g, dev, codes_of(g, N, K), K, block, pow2, cycle([0, -1], K))
    row, col = M - 2, N - 3
    a.scales[row, 1] = float("nan")
    b.scales[col // 128 if block == "tile" else col, -1] = float("nan")
    cols = (torch.arange(N) // 128 == col // 128) if block == "tile" else torch.arange(N) == col
    nan = (torch.arange(M) == row)[:, None] | cols
    if not pow2:
        a.scales[0, 0] = 0.0
        av[0, :128] = 0
    want = torch.mm(av, bv.t().contiguous()).masked_fill(nan.to(dev), 0.0)
    for out, dt in (("bf16", BF16), ("f32", F32)):
        got = dg.block_gemm(a, b, out_dtype=out)
        assert torch.equal(torch.isnan(got).cpu(), nan), out
        bound = product_bound(av, bv, K, want, dt, [])
        assert bool(((got.double().masked_fill(nan.to(dev), 0.0) - want).abs() <= bound).all()), out


@kinds
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_repeat_exactly(dev, M, N, K, block, pow2):
    g = gen(M + N)
    a, _ = operand(g, dev, codes_of(g, M, K), K, "row", pow2, cycle([0, 1], K))
    b, _ = operand(g, dev, codes_of(g, N, K), K, block, pow2, cycle([0, -1], K))
    for out in ("bf16", "f32"):
        first = dg.block_gemm(a, b, out_dtype=out)
        for _ in range(4):
            assert torch.equal(dg.block_gemm(a, b, out_dtype=out), first), out
