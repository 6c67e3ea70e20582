"""The operators around the product against their plain forms in 64 bits."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from dense_gemm_design_amd import ops as O  # noqa: E402
import ops_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = R.U


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load()
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


# ---- quantisation -----------------------------------------------------------------------------

def check_quantize(x_dev, block, side, pow2, what):
    x = x_dev.cpu()
    q = dg.block_quantize(x_dev, block, transposed=side, pow2=pow2)
    got = q if isinstance(q, tuple) else (q,)
    want = [t for t, on in ((x, side is not True), (x.t(), side is not False)) if on]
    assert len(got) == len(want)
    for o, t in zip(got, want):
        codes, scales = R.quantize(t, block, pow2)
        assert o.K == t.shape[1] and o.data.shape == codes.shape and o.scales.shape == scales.shape
        s = o.scales.cpu()
        assert torch.equal(s.isnan(), scales.isnan()), what
        assert torch.equal(s.nan_to_num(0), scales.nan_to_num(0)), what
        c = o.data.cpu()
        # a NaN's sign is nobody's; zeros keep the quotient's
        nan, gnan = (codes & 127) == 127, (c & 127) == 127
        assert torch.equal(nan, gnan), what
        assert torch.equal(c[~nan], codes[~nan]), (what, int((c != codes).sum()))
        assert tuple(o.values.shape) == tuple(t.shape)


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (2, 200), (127, 129), (128, 128),
                                       (130, 16), (300, 257), (515, 1000)])
def test_quantize(dev, rows, cols, dtype, block, pow2):
    print(f"quantize {rows}x{cols} {dtype} {block} pow2={pow2}", flush=True)
    g = gen(rows * 1000 + cols)
    x = (randn(g, rows, cols) * torch.exp(randn(g, rows, 1) * 3)).to(dtype).to(dev)
    for side in (False, True, "both"):
        check_quantize(x, block, side, pow2, f"{rows}x{cols} side {side}")


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantize_values_at_the_edges(dev, dtype, block, pow2):
    """Zeros, infinities, NaN, the smallest and largest magnitudes, quotients on and next to the
    borders between codes."""
    g = gen(5)
    x = randn(g, 260, 520)
    x[0] = 0
    x[1, 130] = float("inf")
    x[2, 5] = float("nan")
    x[3] *= 1e-42
    x[4] *= 1e38 / 6
    x[5] *= 2.0 ** -120
    x[6, :128] = 2.0 ** -149
    x[7] = -0.0
    # borders: amax is 448 (or 7 * 2^k) exactly, the others multiples of half a code's step
    mids = torch.tensor([(a + b) / 2 for a, b in zip(R._POSITIVE, R._POSITIVE[1:])])
    for i, scale in enumerate((1.0, 2.0 ** -9, 3.0, 1.1, 2.0 ** 100)):
        row = torch.cat([mids, torch.tensor([448.0, -448.0])]) * scale
        x[10 + i, :128] = row[:128]
        x[20 + i, 128:256] = torch.nextafter(row[:128], torch.tensor(float("inf")))
        x[30 + i, 128:256] = torch.nextafter(row[:128], torch.tensor(0.0))
        x[20 + i, 255] = x[30 + i, 255] = 448.0 * scale
    x = x.to(dtype).to(dev)
    for side in (False, True, "both"):
        check_quantize(x, block, side, pow2, f"edges side {side}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantize_borders_at_any_scale(dev, dtype):
    """Blocks of every mantissa of amax, filled with numbers next to the borders of its codes."""
    g = gen(6)
    amax = (1 + torch.rand(512, 1, generator=g)).to(dtype).double()
    mids = torch.tensor([(a + b) / 2 for a, b in zip(R._POSITIVE, R._POSITIVE[1:])] + [448.0] * 2)
    x = (mids[None, :128].double() * (amax / 448)).float()
    x = torch.nextafter(x, torch.where(torch.rand(x.shape, generator=g) < 0.5, 0.0, 1e30))
    x[:, 127:] = amax.float()
    check_quantize(x.to(dtype).to(dev), "row", False, False, "borders")
    check_quantize(x.t().contiguous().to(dtype).to(dev), "row", True, False, "borders, transposed")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantize_strided_rows(dev, dtype):
    g = gen(7)
    big = randn(g, 200, 413).to(dtype).to(dev)
    for view in (big[:, 1:301], big[3:133:2, 7:408], big[:1, 5:9].expand(150, 4)):
        check_quantize(view, "row", "both", False, f"stride {view.stride()}")
        check_quantize(view, "tile", "both", True, f"stride {view.stride()}")


def test_quantize_of_nothing(dev):
    q, t = dg.block_quantize(torch.empty(0, 300, device=dev), transposed="both")
    assert q.data.shape == (0, 304) and t.data.shape == (300, 0) and q.scales.shape == (0, 3)


# ---- product ----------------------------------------------------------------------------------

def operand(g, dev, rows, K, block, pow2):
    x = randn(g, rows, K) * torch.exp(randn(g, rows, 1))
    codes, scales = R.quantize(x, block, pow2) if rows * K < 60000 else fast_quantize(x, block, pow2)
    q = dg.BlockScaled(codes.to(dev), scales.t().contiguous().to(dev).t(), K, block, pow2)
    return q, R.spread(codes, scales, block, K)


def fast_quantize(x, block, pow2):
    """Codes and scales of their own, where making them block by block would take long: any will do
    for a product."""
    rows, K = x.shape
    kb = R.up(K, 128)
    sr = R.up(rows, 128) if block == "tile" else rows
    g = gen(rows + 3 * K)
    scales = torch.exp(torch.randn(sr, kb, generator=g) * 0.5)
    if pow2:
        scales = torch.exp2(torch.round(torch.log2(scales)))
    codes = torch.zeros(rows, R.up(K, 16) * 16, dtype=torch.uint8)
    codes[:, :K] = x.clamp(-6, 6).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scales


def fp32_bound(size, K, splits_most=64):
    """Sums in fp32: 128 products of a block in the matrix unit (a step each, not half), the scale's
    two roundings, a half step a block, split and extra.  size: the sum of the terms' magnitudes."""
    return size * ((2 * 128 + 4 + R.up(K, 128) + splits_most + 4) * U)


def aligned_bound(av, bv):
    """What the e4m3 matrix instructions of a bf16 C leave out: of eight neighbouring products seven
    may lose what lies under 2^-13 of the largest."""
    total, top = 0, None
    a, b = av.abs(), bv.abs()
    for k in range(a.shape[1]):
        t = torch.outer(a[:, k], b[:, k])
        top = t if k % 8 == 0 else torch.maximum(top, t)
        if k % 8 == 7 or k == a.shape[1] - 1:
            total = total + top
    return total * (7 * 2.0 ** -13)


def product_bound(av, bv, K, want, out, extras, aligned=None):
    """The sums' error, the extras', and the output's rounding."""
    bound = fp32_bound(torch.mm(av.abs(), bv.abs().t().contiguous()), K)
    if out is BF16:
        bound = bound + (aligned_bound(av, bv) if aligned is None else aligned)
    for e in extras:
        bound = bound + e.abs() * (2 * U)
    return bound + (want.abs() + bound) * R.HALF[out]


SHAPES = [(1, 1, 1), (1, 64, 64), (3, 100, 300), (16, 130, 129), (17, 33, 1000), (32, 256, 2048),
          (33, 64, 128), (100, 250, 1100), (128, 128, 256), (130, 390, 127), (257, 515, 640),
          (300, 129, 4097), (64, 1, 700), (5, 3, 5000)]


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(dev, M, N, K, block, pow2):
    print(f"product {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M * 7 + N * 3 + K)
    a, av = operand(g, dev, M, K, "row", pow2)
    b, bv = operand(g, dev, N, K, block, pow2)
    bias, src = randn(g, N), randn(g, M, N)
    plain = av @ bv.t()
    aligned = aligned_bound(av.to(dev), bv.to(dev)).cpu()
    for out, dt in (("bf16", BF16), ("f32", F32)):
        for kind in ("none", "bias", "source", "bf16 source and bias"):
            kw, extras = {}, []
            if "bias" in kind:
                kw["bias_col"] = bias.to(dev)
                extras.append(bias.double().expand(M, N))
            if "source" in kind:
                s = src.to(BF16) if "bf16" in kind else src
                kw["source"] = s.to(dev)
                extras.append(s.double())
            want = plain + sum(extras) if extras else plain
            got = dg.block_gemm(a, b, out_dtype=out, **kw)
            assert got.dtype is dt
            R.within(got, want, product_bound(av, bv, K, want, dt, extras, aligned), f"{out} {kind}")


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(4100, 4100, 200), (2000, 8200, 384), (70, 5000, 16384),
                                   (1000, 4104, 8201), (2, 16384, 4000)])
def test_product_large(dev, M, N, K, block, pow2):
    print(f"product {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M + N + K)
    a, av = operand(g, dev, M, K, "row", pow2)
    b, bv = operand(g, dev, N, K, block, pow2)
    av, bv = av.to(dev), bv.to(dev)
    bias = randn(g, N).to(dev)
    want = torch.mm(av, bv.t().contiguous()) + bias.double()
    for out, dt in (("bf16", BF16), ("f32", F32)):
        got = dg.block_gemm(a, b, out_dtype=out, bias_col=bias)
        bound = product_bound(av, bv, K, want, dt, [bias.double()])
        bad = ~((got.double() - want).abs() <= bound)
        assert not bool(bad.any()), (out, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(4090, 4104, 100), (4096, 4352, 128), (8200, 2056, 300),
                                   (4090, 4104, 520), (256, 65800, 260)])
def test_product_of_large_tiles(dev, M, N, K, block, pow2):
    """Odd and even counts of k-blocks, one among them, over several tiles a workgroup; edges of
    every kind; rows around C stay as they were."""
    print(f"product {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M + N + K)
    a, av = operand(g, dev, M, K, "row", pow2)
    b, bv = operand(g, dev, N, K, block, pow2)
    av, bv = av.to(dev), bv.to(dev)
    want = torch.mm(av, bv.t().contiguous())
    bound = product_bound(av, bv, K, want, BF16, [])
    for first in (8, 3):          # rows of C at a multiple of 16 bytes, and at 2 bytes
        held = torch.full((N * 16 + M * N,), 5.0, dtype=BF16, device=dev)
        at = N * 8 + (first - 8)
        c = held[at:at + M * N].view(M, N)
        dg.block_gemm(a, b, out=c)
        bad = ~((c.double() - want).abs() <= bound)
        assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())
        assert bool((held[:at] == 5).all()) and bool((held[at + M * N:] == 5).all())


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(66000, 1, 130), (65600, 3, 200), (65700, 6, 100), (4099, 4201, 130),
                                   (700, 903, 128), (129, 2, 4000), (256, 5, 300)])
@pytest.mark.parametrize("source", [BF16, F32], ids=["bf16", "f32"])
def test_product_with_extras(dev, M, N, K, block, pow2, source):
    """Bias and source with rows that end inside four columns, and fewer columns than that."""
    print(f"product {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M + N + K)
    a, av = operand(g, dev, M, K, "row", pow2)
    b, bv = operand(g, dev, N, K, block, pow2)
    av, bv = av.to(dev), bv.to(dev)
    bias, src = randn(g, N).to(dev), randn(g, M, N).to(source).to(dev)
    extras = [bias.double(), src.double()]
    want = torch.mm(av, bv.t().contiguous()) + extras[0] + extras[1]
    for dt in (BF16, F32):
        bound = product_bound(av, bv, K, want, dt, extras)
        whole = torch.full((M + 2, N), 7.0, dtype=dt, device=dev)
        for into in (False, True):   # and into the source itself, where types allow
            if into and dt is not source:
                continue
            if into:
                whole[1:-1] = src
            dg.block_gemm(a, b, bias_col=bias, source=whole[1:-1] if into else src, out=whole[1:-1])
            bad = ~((whole[1:-1].double() - want).abs() <= bound)
            assert not bool(bad.any()), (dt, into, int(bad.sum()), bad.nonzero()[0].tolist())
            assert bool((whole[0] == 7).all()) and bool((whole[-1] == 7).all())


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(2171, 2045, 4300), (140, 139, 16000), (1300, 1300, 1100),
                                   (33, 4300, 3700)])
def test_product_of_cut_tiles(dev, M, N, K, block, pow2):
    """Few tiles of much K, and some over what fills the chip: pieces of odd and even length, edges in
    them, and all that is added behind them; memory around C stays as it was."""
    print(f"product {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    g = gen(M + N + K)
    a, av = operand(g, dev, M, K, "row", pow2)
    b, bv = operand(g, dev, N, K, block, pow2)
    av, bv = av.to(dev), bv.to(dev)
    bias, src = randn(g, N).to(dev), randn(g, M, N).to(BF16).to(dev)
    extras = [bias.double(), src.double()]
    want = torch.mm(av, bv.t().contiguous()) + extras[0] + extras[1]
    for dt in (BF16, F32):
        whole = torch.full((M + 2, N), 7.0, dtype=dt, device=dev)
        dg.block_gemm(a, b, bias_col=bias, source=src, out=whole[1:-1])
        bound = product_bound(av, bv, K, want, dt, extras)
        bad = ~((whole[1:-1].double() - want).abs() <= bound)
        assert not bool(bad.any()), (dt, int(bad.sum()), bad.nonzero()[0].tolist())
        assert bool((whole[0] == 7).all()) and bool((whole[-1] == 7).all())
        again = torch.empty(M, N, dtype=dt, device=dev)
        dg.block_gemm(a, b, bias_col=bias, source=src, out=again)
        assert torch.equal(again, whole[1:-1]), "sums in another order"


def test_product_adds_into_its_source(dev):
    g = gen(11)
    for M, N, K in ((20, 70, 300), (200, 70, 300), (64, 130, 9000)):
        a, av = operand(g, dev, M, K, "row", False)
        b, bv = operand(g, dev, N, K, "row", False)
        c = randn(g, M, N).to(dev)
        want = av @ bv.t() + c.double().cpu()
        bound = product_bound(av, bv, K, want, F32, [c.double().cpu()])
        got = dg.block_gemm(a, b, source=c, out=c)
        assert got is c
        R.within(c, want, bound, f"{M}x{N}x{K}")


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
def test_product_of_a_block_that_is_not_a_number(dev, pow2):
    """An infinity in one block of A makes its row NaN and no other."""
    for M in (8, 150):
        g = gen(12)
        x = randn(g, M, 500)
        x[3, 200] = float("inf")
        b, _ = operand(g, dev, 90, 500, "tile", pow2)
        a = dg.block_quantize(x.to(dev), "row", pow2=pow2)
        nan = torch.isnan(dg.block_gemm(a, b, out_dtype="f32")).cpu()
        assert bool(nan[3].all()) and int(nan.sum()) == 90


def test_product_without_columns_is_its_extras(dev):
    a = dg.BlockScaled(torch.empty(40, 0, dtype=torch.uint8, device=dev),
                       torch.empty(40, 0, device=dev), 0, "row")
    b = dg.BlockScaled(torch.empty(30, 0, dtype=torch.uint8, device=dev),
                       torch.empty(30, 0, device=dev), 0, "row")
    src = randn(gen(1), 40, 30).to(dev)
    assert torch.equal(dg.block_gemm(a, b, out_dtype="f32", source=src), src)
    assert dg.block_gemm(dg.BlockScaled(a.data[:0], a.scales[:0], 0, "row"), b).shape == (0, 30)


def test_product_of_wider_storage(dev):
    """Operands that are slices of wider matrices: what lies between rows and blocks is not read."""
    g = gen(13)
    for M, N in ((9, 40), (140, 200)):
        K = 400
        a, av = operand(g, dev, M, K, "row", False)
        b, bv = operand(g, dev, N, K, "row", False)
        want = av @ bv.t()
        wide = []
        for q in (a, b):
            data = torch.full((q.data.shape[0], 512), 0x7F, dtype=torch.uint8, device=dev)
            data[:, :400] = q.data
            scales = torch.full((4, q.scales.shape[0] + 5), float("nan"), device=dev)
            scales[:, :q.scales.shape[0]] = q.scales.t()
            wide.append(dg.BlockScaled(data[:, :400], scales[:, :q.scales.shape[0]].t(), K, "row"))
        got = dg.block_gemm(*wide, out_dtype="f32")
        R.within(got, want, product_bound(av, bv, K, want, F32, []), f"{M}x{N}")


# ---- layer norm -------------------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (1, 5), (3, 64), (5, 1111), (7, 512), (9, 513), (130, 1000), (33, 2048),
               (4, 2049), (2100, 72), (17, 4096), (3, 4100), (6, 8192), (2, 9001), (3, 16384),
               (2, 16385), (2, 40003)]


def norm_inputs(g, dev, rows, cols, dtype, wtype):
    x = (randn(g, rows, cols) * torch.exp(randn(g, rows, 1)) + randn(g, rows, 1)).to(dtype)
    w, b = (1 + 0.2 * randn(g, cols)).to(wtype), (0.3 * randn(g, cols)).to(wtype)
    return x.to(dev), w.to(dev), b.to(dev)


def steps_of(cols):
    """Additions that a value of a row passes through: a thread's own, then the tree's."""
    return max(32, R.up(cols, 1024) + 8) + 24


def check_norm(x, w, b, eps, what):
    y, mean, rstd = dg.layer_norm(x, w, b, eps=eps)
    X, W = x.cpu().double(), w.cpu().double()
    want, wm, wr = R.norm(x.cpu(), w.cpu(), b.cpu() if b is not None else None, eps)
    n = steps_of(x.shape[1])
    dm = n * U * X.abs().mean(1)                        # the mean's error
    d = (X - wm[:, None]).abs()
    # d's own error enters the variance twice; then its sum and the root
    dr = wr * (wr * wr * (d * (dm[:, None] + U * d)).mean(1) * 2 + n * U + (dm * wr) ** 2)
    R.within(mean, wm, dm + U * wm.abs(), what + " mean")
    R.within(rstd, wr, dr + 2 * U * wr, what + " rstd")
    h = d * wr[:, None]
    bound = W.abs() * (dm * wr)[:, None] + W.abs() * d * dr[:, None] + 4 * U * h * W.abs()
    bound = bound + 2 * U * want.abs() + (b.cpu().double().abs() * U if b is not None else 0)
    R.within(y, want, bound + (want.abs() + bound) * R.HALF[x.dtype], what + " y")


@pytest.mark.parametrize("types", [(BF16, F32), (BF16, BF16), (F32, F32)],
                         ids=["bf16-f32", "bf16-bf16", "f32-f32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_layer_norm(dev, rows, cols, types):
    print(f"layer norm {rows}x{cols} {types}", flush=True)
    x, w, b = norm_inputs(gen(rows + cols), dev, rows, cols, *types)
    check_norm(x, w, b, 1e-5, f"{rows}x{cols}")
    check_norm(x, w, None, 1e-2, f"{rows}x{cols} without bias")


def grad_bounds(dy, x, w, mean, rstd):
    dy, x, w, mean, rstd = (t.double().cpu() for t in (dy, x, w, mean, rstd))
    rows, cols = x.shape
    n = steps_of(cols) + 8
    h = ((x - mean[:, None]) * rstd[:, None]).abs()
    g = (dy * w).abs()
    dx = rstd[:, None] * (g + g.mean(1, keepdim=True) + h * (g * h).mean(1, keepdim=True)) * (n * U)
    return dx, (dy.abs() * h).sum(0) * ((rows + 80) * U), dy.abs().sum(0) * ((rows + 80) * U)


def check_norm_grad(dy, x, w, what):
    _, mean, rstd = dg.layer_norm(x, w, None)
    got = dg.layer_norm_backward(dy, x, w, mean, rstd)
    want = R.norm_grad(*(t.cpu() for t in (dy, x, w, mean, rstd)))
    for o, t, e, name in zip(got, want, grad_bounds(dy, x, w, mean, rstd), ("dx", "dw", "db")):
        R.within(o, t, e + (t.abs() + e) * R.HALF[o.dtype], f"{what} {name}")


@pytest.mark.parametrize("types", [(BF16, F32), (BF16, BF16), (F32, F32)],
                         ids=["bf16-f32", "bf16-bf16", "f32-f32"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(1500, 136), (700, 4096), (600, 16400)])
def test_layer_norm_backward(dev, rows, cols, types):
    print(f"layer norm backward {rows}x{cols} {types}", flush=True)
    g = gen(rows + 2 * cols)
    x, w, _ = norm_inputs(g, dev, rows, cols, *types)
    dy = (0.1 * randn(g, rows, cols)).to(types[0]).to(dev)
    check_norm_grad(dy, x, w, f"{rows}x{cols}")


@pytest.mark.parametrize("types", [(BF16, F32), (BF16, BF16), (F32, F32)],
                         ids=["bf16-f32", "bf16-bf16", "f32-f32"])
@pytest.mark.parametrize("rows,cols", [(15, 17), (17, 15), (64, 500), (65, 520), (255, 2050), (257, 33),
                                       (515, 1111), (576, 2048), (577, 2048), (575, 1025), (580, 900),
                                       (600, 3000), (576, 4097)])
def test_layer_norm_backward_of_few_rows(dev, rows, cols, types):
    print(f"layer norm backward {rows}x{cols} {types}", flush=True)
    g = gen(rows + 2 * cols)
    x, w, _ = norm_inputs(g, dev, rows, cols, *types)
    dy = randn(g, rows, cols).to(types[0]).to(dev)
    check_norm_grad(dy, x, w, f"{rows}x{cols}")
    if rows <= 100:
        wide = randn(g, rows, 2 * cols + 3).to(types[0]).to(dev)
        check_norm_grad(dy[:1].expand(rows, cols), wide[:, 1:cols + 1], w, f"{rows}x{cols} strided")


def test_layer_norm_backward_over_its_inputs(dev):
    """dx may be written over dy or x through the C ABI."""
    lib = O.load()
    g = gen(41)
    for rows, cols in ((40, 300), (300, 1500)):
        x, w, _ = norm_inputs(g, dev, rows, cols, F32, F32)
        dy = randn(g, rows, cols).to(dev)
        _, mean, rstd = dg.layer_norm(x, w, None)
        want = R.norm_grad(*(t.cpu() for t in (dy, x, w, mean, rstd)))
        bounds = grad_bounds(dy, x, w, mean, rstd)
        n = ctypes.c_size_t()
        assert lib.gemm_layer_norm_backward_workspace(rows, cols, ctypes.byref(n)) == 0
        work = torch.empty(n.value, dtype=torch.uint8, device=dev)
        for over in ("dy", "x"):
            d, v = dy.clone(), x.clone()
            dx = d if over == "dy" else v
            dw, db = torch.empty(cols, device=dev), torch.empty(cols, device=dev)
            st = lib.gemm_layer_norm_backward(
                d.data_ptr(), cols, v.data_ptr(), cols, 2, rows, cols, w.data_ptr(), 2,
                mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
                work.data_ptr(), n.value, torch.cuda.current_stream().cuda_stream)
            assert st == 0
            for o, t, e, name in zip((dx, dw, db), want, bounds, ("dx", "dw", "db")):
                R.within(o, t, e + (t.abs() + e) * R.HALF[F32], f"over {over} {name}")


def test_layer_norm_strided_rows(dev):
    g = gen(21)
    big, bigd = (randn(g, 60, 1501).to(BF16).to(dev) for _ in range(2))
    w, b = randn(g, 700).to(dev), randn(g, 700).to(dev)
    for at in (0, 1, 3):
        x, dy = big[::2, at:at + 700], bigd[30:, at + 2:at + 702]
        check_norm(x, w, b, 1e-5, f"offset {at}")
        check_norm_grad(dy, x, w, f"offset {at}")
    # one row's gradient for every row: a stride of zero
    check_norm_grad(bigd[:1, :700].expand(60, 700), big[:, :700], w, "broadcast gradient")


def test_layer_norm_rows_of_one_value(dev):
    """A row of one value has no spread: y is the bias, and rstd 1 / sqrt(eps)."""
    x = torch.full((3, 200), 2.0, device=dev)
    b = randn(gen(2), 200).to(dev)
    y, mean, rstd = dg.layer_norm(x, torch.ones(200, device=dev), b, eps=1e-4)
    assert torch.equal(y, b.expand(3, 200)) and bool((mean == 2).all())
    assert bool(((rstd - 100).abs() < 1e-4).all())


def test_layer_norm_row_with_an_infinity(dev):
    """It spoils its own row, and the weight's gradients, alone."""
    x = randn(gen(3), 6, 300).to(dev)
    x[2, 7] = float("inf")
    y, mean, rstd = dg.layer_norm(x, torch.ones(300, device=dev))
    bad = ~torch.isfinite(y)
    assert bool(bad[2].any()) and not bool(bad[[0, 1, 3, 4, 5]].any())


def test_layer_norm_of_no_rows(dev):
    w = torch.ones(70, device=dev)
    y, mean, rstd = dg.layer_norm(torch.empty(0, 70, device=dev), w, w)
    assert y.shape == (0, 70) and mean.shape == rstd.shape == (0,)
    dx, dw, db = dg.layer_norm_backward(y, y, w, mean, rstd)
    assert dx.shape == (0, 70) and not bool(dw.any()) and not bool(db.any())


def test_layer_norm_gradient_against_differences(dev):
    """Along random directions, the central difference of the 64-bit norm (step 1e-5: its own error
    is under 1e-8 of the terms' size) against the kernel's gradient."""
    g = gen(22)
    rows, cols, eps, step = 40, 333, 1e-5, 1e-5
    x, w, b = norm_inputs(g, dev, rows, cols, F32, F32)
    dy = randn(g, rows, cols).to(dev)
    _, mean, rstd = dg.layer_norm(x, w, b, eps=eps)
    dx, dw, db = (t.double().cpu() for t in dg.layer_norm_backward(dy, x, w, mean, rstd))
    ex, ew, eb = grad_bounds(dy, x, w, mean, rstd)
    X, W, B, DY = (t.double().cpu() for t in (x, w, b, dy))

    def loss(x_, w_, b_):
        return float((R.norm(x_, w_, b_, eps)[0] * DY).sum())

    size = float((R.norm(X, W, B, eps)[0].abs() * DY.abs()).sum())
    # mean and rstd are rounded to fp32 before the gradient uses them: 2^-24 of each term, and n
    # such roundings inside them (steps_of), as bounds on the gradient's terms
    slack = 4 * steps_of(cols)
    for k in range(4):
        v, vw, vb = randn(g, rows, cols).double(), randn(g, cols).double(), randn(g, cols).double()
        for grad, err, move, args in (
                (dx, ex, v, lambda s: (X + s * v, W, B)), (dw, ew, vw, lambda s: (X, W + s * vw, B)),
                (db, eb, vb, lambda s: (X, W, B + s * vb))):
            diff = (loss(*args(step)) - loss(*args(-step))) / (2 * step)
            bound = float((err * move.abs()).sum()) * slack / 8 + size * 1e-7
            assert abs(diff - float((grad * move).sum())) <= bound


# ---- clipping ---------------------------------------------------------------------------------

def some_gradients(g, dev, sizes):
    return [(randn(g, n) * 0.1).to(BF16 if i % 3 else F32).to(dev) for i, n in enumerate(sizes)]


def check_clip(grads, max_norm, into, what):
    before = [t.clone() for t in grads]
    out = [torch.full_like(t, 9.0) for t in grads] if into else None
    want = sum(float((t.double() ** 2).sum()) for t in before) ** 0.5
    alone = dg.grad_norm(grads)
    norm = dg.clip_grad_norm(grads, max_norm, out=out)
    assert norm.shape == () and norm.dtype is F32 and torch.equal(alone, norm)
    assert abs(float(norm) - want) <= 2 * U * want, what
    c = min(1.0, max_norm / (want + 1e-6))
    for o, t in zip(out if into else grads, before):
        v = t.double().cpu() * c
        R.within(o, v, v.abs() * (6 * U) + v.abs() * R.HALF[t.dtype], what)
        if into:
            continue
        if c == 1.0:
            assert torch.equal(o, t)
    if into:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("into", [False, True], ids=["in_place", "into"])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 3], [16384, 16385, 5, 100000], [33] * 300,
                                   [3000001, 1, 640000]], ids=["one", "small", "chunks", "many",
                                                              "large"])
def test_clip(dev, sizes, into):
    print(f"clip {sizes[:4]} into={into}", flush=True)
    g = gen(len(sizes) + sizes[0])
    for max_norm in (1e-2, 1e6):
        check_clip(some_gradients(g, dev, sizes), max_norm, into, f"{max_norm}")


def test_clip_at_any_alignment(dev):
    g = gen(31)
    flat, flat32 = randn(g, 50000).to(BF16).to(dev), randn(g, 50000).to(dev)
    grads = [flat[1:20000], flat32[3:17000], flat[20001:20008], flat32[17001:40000].view(-1, 1)]
    check_clip(grads, 0.5, False, "views")
    check_clip(grads, 0.5, True, "views")
    assert float(flat[20000]) == float(flat[20000]) and bool(torch.isfinite(flat32).all())


@pytest.mark.parametrize("into", [False, True], ids=["in_place", "into"])
def test_clip_of_a_list_longer_than_the_caches(dev, into):
    torch.manual_seed(32)
    grads = [(torch.randn(n, device=dev) * 0.1).to(t)
             for n, t in ((20_000_003, BF16), (12_345_677, F32), (17, BF16), (9_000_000, F32))]
    before = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads] if into else None
    want = sum(float((t.double() ** 2).sum()) for t in before) ** 0.5
    norm = dg.clip_grad_norm(grads, 0.5, out=out)
    assert abs(float(norm) - want) <= 2 * U * want
    for o, t in zip(out or grads, before):
        v = t.double() * (0.5 / (want + 1e-6))
        assert bool(((o.double() - v).abs() <= v.abs() * (6 * U + R.HALF[t.dtype])).all())


def test_clip_of_large_squares_and_of_nothing(dev):
    big = [torch.full((1000,), 1e30, device=dev)]
    want = 1e30 * 1000 ** 0.5
    assert abs(float(dg.grad_norm(big)) / want - 1) < 1e-6
    zero = [torch.zeros(100, device=dev), torch.zeros(0, device=dev)]
    assert float(dg.clip_grad_norm(zero, 1.0)) == 0.0 and not bool(zero[0].any())
    assert float(dg.clip_grad_norm([zero[1]], 1.0)) == 0.0


def test_clip_of_what_is_not_finite(dev):
    """An infinite norm scales by zero, a NaN makes everything NaN."""
    a, b = torch.ones(50, device=dev), torch.ones(20000, device=dev, dtype=BF16)
    b[10000] = float("inf")
    assert float(dg.clip_grad_norm([a, b], 1.0)) == float("inf")
    assert not bool(a.any()) and bool(torch.isnan(b[10000])) and int(torch.isnan(b).sum()) == 1
    a.fill_(1.0)[3] = float("nan")
    c = torch.ones(5, device=dev)
    assert bool(torch.isnan(dg.clip_grad_norm([a, c], 1.0)))
    assert bool(torch.isnan(a).all()) and bool(torch.isnan(c).all())


# ---- streams and graphs -----------------------------------------------------------------------

def whole_step(x, w, b, wq, dy):
    y, mean, rstd = dg.layer_norm(x, w, b)
    q, qt = dg.block_quantize(y, "row", transposed="both")
    c = dg.block_gemm(q, wq, out_dtype="f32")
    few = dg.block_gemm(dg.BlockScaled(q.data[:4], q.scales[:4], q.K, "row"), wq)
    dyq, dyt = dg.block_quantize(dy, "row", transposed="both")
    dwq = dg.block_gemm(dyt, qt, out_dtype="f32")
    dx, dw, db = dg.layer_norm_backward(y, x, w, mean, rstd)
    out = [torch.empty_like(t) for t in (dwq, dx, dw, db)]
    norm = dg.clip_grad_norm([dwq, dx, dw, db], 0.1, out=out)
    return [y, mean, rstd, q.data, qt.data, c, few, dwq, dx, dw, db, norm, *out]


def step_inputs(dev, seed):
    g = gen(seed)
    x = randn(g, 300, 520).to(BF16).to(dev)
    w, b = randn(g, 520).to(dev), randn(g, 520).to(dev)
    wq = dg.block_quantize(randn(g, 200, 520).to(dev), "tile")
    return x, w, b, wq, randn(g, 300, 200).to(BF16).to(dev)


def test_graph_replays_give_what_eager_calls_give(dev):
    x, w, b, wq, dy = step_inputs(dev, 41)
    for _ in range(2):
        whole_step(x, w, b, wq, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = whole_step(x, w, b, wq, dy)
    for seed in (41, 42, 43):
        nx, _, _, _, ndy = step_inputs(dev, seed)
        x.copy_(nx)
        dy.copy_(ndy)
        eager = [t.clone() for t in whole_step(x, w, b, wq, dy)]
        for t in held:
            t.view(torch.uint8).fill_(0x55) if t.dim() else t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (s, t) in enumerate(zip(held, eager)):
            assert torch.equal(s, t), (seed, i)


def test_other_streams_give_the_same(dev):
    x, w, b, wq, dy = step_inputs(dev, 44)
    want = whole_step(x, w, b, wq, dy)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(whole_step(x, w, b, wq, dy))
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        for i, (s, t) in enumerate(zip(outs, want)):
            assert torch.equal(s, t), (k, i)
