"""int8 quantisation a row and the product of its operands against plain forms in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from test_gpu_ops import dev, gen, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = R.U
TYPES = [BF16, F32]
NAMES = ["bf16", "f32"]


# ---- quantisation -----------------------------------------------------------------------------

def plain_quantize(x):
    """(codes, scales) of a CPU tensor.  amax / 127 in fp64 is no fp32 midpoint (it would be one of
    127ths), and the quotient of two fp32 numbers is 2^-49 away from a border or on it: so both are the exact
    value's roundings."""
    amax = x.abs().amax(dim=1).double()
    scales = (amax / 127).float().clamp(min=2.0 ** -120)
    fine = torch.isfinite(amax)
    codes = torch.round(torch.where(fine[:, None], x.double(), 0.0) / scales.double()[:, None])
    codes = torch.where(fine[:, None], codes, torch.zeros_like(codes)).to(torch.int8)
    return codes, torch.where(fine, scales, torch.full_like(scales, float("nan")))


def check_quantize(x_dev, side, what):
    x = x_dev.cpu()
    q = dg.int8_quantize(x_dev, transposed=side)
    got = q if isinstance(q, tuple) else (q,)
    want = [t for t, on in ((x, side is not True), (x.t(), side is not False)) if on]
    assert len(got) == len(want)
    for o, t in zip(got, want):
        codes, scales = plain_quantize(t)
        rows, cols = t.shape
        assert o.K == cols and o.scales.shape == (rows,) and o.data.shape == (rows, R.up(cols, 16) * 16)
        s = o.scales.cpu()
        assert torch.equal(s.isnan(), scales.isnan()), what
        assert torch.equal(s.nan_to_num(0), scales.nan_to_num(0)), what
        c = o.data.cpu()
        assert torch.equal(c[:, :cols], codes), (what, int((c[:, :cols] != codes).sum()))
        assert not bool(c[:, cols:].any()), what
        assert torch.equal(o.values, o.data[:, :cols])


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (2, 200), (127, 129), (128, 128), (130, 16),
                                       (300, 257), (515, 1000), (3, 1025), (5, 2049), (9, 4097),
                                       (2, 9000), (3, 17000), (2, 40001), (1, 65536), (2, 65537),
                                       (3, 70001), (5000, 24), (9000, 130), (70, 20000), (2049, 130),
                                       (2048, 40), (2047, 2100), (1024, 4000), (1009, 60), (513, 17),
                                       (512, 300), (511, 2050), (3000, 3001), (6000, 1500)])
def test_quantize(dev, rows, cols, dtype):
    print(f"int8 quantize {rows}x{cols} {dtype}", flush=True)
    g = gen(rows * 1000 + cols)
    x = (randn(g, rows, cols) * torch.exp(randn(g, rows, 1) * 3)).to(dtype).to(dev)
    for side in (False, True, "both"):
        check_quantize(x, side, f"{rows}x{cols} side {side}")


@pytest.mark.parametrize("rows,cols", [(60, 300), (60, 1500), (60, 9000), (600, 300), (1500, 300), (2200, 300)])
@pytest.mark.parametrize("dtype", TYPES, ids=NAMES)
def test_quantize_values_at_the_edges(dev, dtype, rows, cols):
    """Zeros, infinities, NaN, the smallest and largest magnitudes, ties and what lies next to them."""
    g = gen(5)
    x = randn(g, rows, cols)
    x[0] = 0
    x[1, 130] = float("inf")
    x[2, 5] = float("nan")
    x[3] *= 1e-42
    x[4] *= 1e38 / 6
    x[5] *= 2.0 ** -118
    x[6, :128] = 2.0 ** -149
    x[7] = -0.0
    x[8, 17] = float("-inf")
    ties = torch.arange(-126, 127).float() + 0.5
    for i, scale in enumerate((1.0, 2.0 ** -9, 3.0, 1.1, 2.0 ** 100, 2.0 ** -119)):
        row = torch.cat([ties, torch.tensor([127.0, -127.0])]) * scale
        x[10 + i, :255] = row
        x[20 + i, :255] = torch.nextafter(row, torch.tensor(float("inf")))
        x[30 + i, :255] = torch.nextafter(row, torch.tensor(0.0))
        x[20 + i, 255:] = x[30 + i, 255:] = 0
        x[20 + i, 256] = x[30 + i, 256] = 127.0 * scale
    x = x.to(dtype).to(dev)
    for side in (False, True, "both"):
        check_quantize(x, side, f"edges side {side}")


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES)
def test_quantize_ties_at_any_scale(dev, dtype):
    """Rows of every kind of mantissa of amax, filled with the numbers nearest to the borders of its codes."""
    g = gen(6)
    amax = (1 + torch.rand(2048, 1, generator=g)).to(dtype).double()
    ties = (torch.arange(-126, 127).double() + 0.5)[None, :]
    x = (ties * (amax / 127)).float()
    step = torch.randint(-1, 2, x.shape, generator=g).float()
    x = torch.where(step == 0, x, torch.nextafter(x, step * 1e30))
    x = torch.cat([x, amax.float(), -amax.float() / 2], dim=1).to(dtype)
    check_quantize(x.to(dev), False, "ties")
    check_quantize(x.t().contiguous().to(dev), True, "ties, transposed")
    check_quantize(x.t().repeat(4, 1).to(dev), True, "ties, transposed, in sixteen waves")
    check_quantize(x.t().repeat(9, 1).to(dev), True, "ties, transposed, in tiles")


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES)
def test_quantize_strided_rows(dev, dtype):
    big = randn(gen(7), 2500, 413).to(dtype).to(dev)
    for view in (big[:200, 1:301], big[3:133:2, 7:408], big[:1, 5:9].expand(150, 4), big[:, 1:301],
                 big[:1500, 3:400], big[:1, 5:9].expand(2300, 4)):
        for side in (False, True, "both"):
            check_quantize(view, side, f"stride {view.stride()} {side}")


def test_quantize_of_nothing(dev):
    q, t = dg.int8_quantize(torch.empty(0, 300, device=dev), transposed="both")
    assert q.data.shape == (0, 304) and q.scales.shape == (0,)
    assert t.data.shape == (300, 0) and t.K == 0 and bool((t.scales == 2.0 ** -120).all())
    q = dg.int8_quantize(torch.empty(3, 0, device=dev))
    assert q.data.shape == (3, 0) and bool((q.scales == 2.0 ** -120).all())


# ---- product ----------------------------------------------------------------------------------

def operand(g, rows, K, dev, least=-127):
    """Codes of the whole range with rows of their own size, and scales."""
    data = torch.zeros(rows, R.up(K, 16) * 16, dtype=torch.int8)
    data[:, :K] = torch.randint(least, 128, (rows, K), generator=g, dtype=torch.int8)
    scales = torch.exp(randn(g, rows)) * 1e-2
    return dg.Int8Scaled(data.to(dev), scales.to(dev), K)


def sums(a, b):
    """The exact sums, as float64 (they are whole numbers under 2^53)."""
    x, y = a.values.double(), b.values.double()
    if x.is_cuda:
        return torch.mm(x, y.t().contiguous()).cpu()
    return x @ y.t()


def check_product(a, b, out, what, bias=None, source=None, into=None):
    got = dg.int8_gemm(a, b, out_dtype="bf16" if out == BF16 else "f32", bias_col=bias, source=source,
                       out=into)
    t = sums(a, b) * a.scales.cpu().double()[:, None] * b.scales.cpu().double()
    z = t if bias is None else t + bias.cpu().double()
    want = z if source is None else z + source.cpu().double()
    # the sum, its product with one scale, the next product with the bias added, the source added
    bound = 2 * U * t.abs() + U * z.abs() + R.HALF[out] * want.abs() * (1 + 4 * U) + 2.0 ** -148
    if source is not None:
        bound += U * want.abs()
    assert got.dtype == out
    R.within(got, want, bound * (1 + 2.0 ** -20), what)
    return got


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 3, 200), (2, 130, 100), (5, 70, 1), (16, 16, 16), (17, 40, 300),
          (32, 129, 500), (33, 257, 129), (64, 200, 1000), (65, 2, 128), (70, 300, 257), (128, 128, 128),
          (129, 130, 640), (200, 515, 1111), (300, 1, 300), (256, 256, 4096), (1, 5000, 2048),
          (40, 100, 9000), (100, 90, 20000), (513, 1030, 272)]


@pytest.mark.parametrize("out", TYPES, ids=NAMES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(dev, M, N, K, out):
    print(f"int8 product {M}x{N}x{K} {out}", flush=True)
    g = gen(M * 7 + N * 3 + K)
    a, b = operand(g, M, K, dev), operand(g, N, K, dev)
    check_product(a, b, out, "plain")
    check_product(a, b, out, "bias", bias=randn(g, N).to(dev))


@pytest.mark.parametrize("source", TYPES, ids=NAMES)
@pytest.mark.parametrize("out", TYPES, ids=NAMES)
@pytest.mark.parametrize("M,N,K", [(1, 64, 300), (3, 3, 50), (33, 130, 200), (70, 2, 400),
                                   (130, 257, 300), (300, 200, 70), (60, 100, 5000), (90, 130, 9000)])
def test_product_with_extras(dev, M, N, K, out, source):
    g = gen(M + N + K)
    a, b = operand(g, M, K, dev), operand(g, N, K, dev)
    bias, src = randn(g, N).to(dev) * 100, (randn(g, M, N) * 100).to(source).to(dev)
    check_product(a, b, out, "source", source=src)
    check_product(a, b, out, "both", bias=bias, source=src)
    into = torch.empty(M, N, dtype=out, device=dev)
    got = check_product(a, b, out, "into", bias=bias, source=src, into=into)
    assert got.data_ptr() == into.data_ptr()
    if source == out:   # the source itself
        held = src.clone()
        assert torch.equal(dg.int8_gemm(a, b, bias_col=bias, source=held, out=held), got)


LARGE = [(2048, 4096, 1024), (4096, 2304, 384), (1000, 4104, 2001), (300, 8192, 4096), (6000, 1111, 130),
         (64, 14336, 512), (2561, 4000, 257), (4096, 4096, 128), (4100, 4098, 250), (3840, 5376, 300)]


@pytest.mark.parametrize("out", TYPES, ids=NAMES)
@pytest.mark.parametrize("M,N,K", LARGE)
def test_product_large(dev, M, N, K, out):
    print(f"int8 product {M}x{N}x{K} {out}", flush=True)
    g = gen(M + N + K)
    a, b = operand(g, M, K, dev), operand(g, N, K, dev)
    bias = randn(g, N).to(dev)
    check_product(a, b, out, "bias", bias=bias)
    src = randn(g, M, N).to(dev)
    got = check_product(a, b, out, "source", source=src)
    if out == F32:   # the source itself
        assert torch.equal(dg.int8_gemm(a, b, source=src, out=src), got)
    else:
        src = src.to(BF16)
        got = check_product(a, b, out, "bf16 source", bias=bias, source=src)
        assert torch.equal(dg.int8_gemm(a, b, bias_col=bias, source=src, out=src), got)


@pytest.mark.parametrize("M,N,K", [(3, 20, 131071), (3, 20, 131072), (40, 70, 262145), (130, 140, 140000),
                                   (300, 260, 200000)])
def test_product_of_long_sums(dev, M, N, K):
    """Sums past 2^31: all codes -128 give the largest."""
    print(f"int8 product {M}x{N}x{K}", flush=True)
    g = gen(K)
    a, b = operand(g, M, K, dev, -128), operand(g, N, K, dev, -128)
    a.data[0, :K] = b.data[0, :K] = -128
    a.data[-1, :K] = 127
    got = check_product(a, b, F32, "long")
    assert abs(float(got[0, 0]) / (float(a.scales[0]) * float(b.scales[0]) * 2.0 ** 14 * K) - 1) < 4 * U


def test_product_of_long_sums_and_many_tiles(dev):
    """K in five pieces, and more tiles than there is room for at six."""
    M, N, K = 1900, 2000, 540000
    g = torch.Generator(device=dev).manual_seed(12)
    a, b = (dg.Int8Scaled(torch.randint(-128, 128, (rows, K), generator=g, device=dev, dtype=torch.int8),
                          torch.rand(rows, generator=g, device=dev) + 0.5, K) for rows in (M, N))
    a.data[:40] = b.data[:40] = -128
    check_product(a, b, F32, "long and many")


def test_product_is_the_same_in_every_batch(dev):
    """Sums are exact, and the rest is element by element: a row has the same bits alone and in any batch,
    and a column in any weight."""
    g = gen(11)
    K = 1111
    a, b = operand(g, 4100, K, dev), operand(g, 4100, K, dev)
    part = lambda q, n: dg.Int8Scaled(q.data[:n], q.scales[:n], K)   # noqa: E731
    for out in ("f32", "bf16"):
        whole = dg.int8_gemm(a, b, out_dtype=out)
        for M, N in ((1, 4100), (20, 4100), (60, 4096), (100, 300), (1000, 4100), (2048, 1024), (4096, 4097),
                     (4100, 3), (300, 17)):
            assert torch.equal(dg.int8_gemm(part(a, M), part(b, N), out_dtype=out), whole[:M, :N]), (M, N)


@pytest.mark.parametrize("M,N", [(4, 40), (40, 70), (100, 200), (4096, 4352)])
def test_product_with_scales_of_any_size(dev, M, N):
    """Neither a scale times the sum nor the scales' product may leave fp32's range where C does not."""
    g = gen(12)
    K = 200
    a, b = operand(g, M, K, dev), operand(g, N, K, dev)
    b.data[1, :] = 0
    for ea, eb in ((120, -130), (-130, 120), (-100, 100), (100, -120), (60, 60), (-70, -70), (127, -149),
                   (91, -149), (-149, 100), (0, -149)):
        a.scales.copy_(torch.ldexp(1 + torch.rand(M, generator=g), torch.tensor(ea)).clamp(max=3e38))
        b.scales.copy_(torch.ldexp(1 + torch.rand(N, generator=g), torch.tensor(eb)).clamp(max=3e38))
        a.scales[1] = 1.5
        for out in TYPES:
            if out == BF16 and ea + eb < -120:
                continue   # (results under bf16's smallest normal number: another rounding)
            got = dg.int8_gemm(a, b, out_dtype="f32" if out == F32 else "bf16").double().cpu()
            want = sums(a, b) * a.scales.cpu().double()[:, None] * b.scales.cpu().double()
            bound = (3 * U + R.HALF[out]) * want.abs() * (1 + 2.0 ** -20) + 2.0 ** -133 * (out == BF16) \
                + 2.0 ** -148
            fine = want.abs() < 3.3e38
            assert bool(((got - want).abs()[fine] <= bound[fine]).all()), (ea, eb, out)
            assert bool((got[want.abs() > 3.5e38].abs() == float("inf")).all()), (ea, eb, out)


@pytest.mark.parametrize("M,N", [(4, 40), (100, 200), (4096, 4352)])
def test_product_of_a_row_that_is_not_a_number(dev, M, N):
    g = gen(13)
    x, y = randn(g, M, 300), randn(g, N, 300)
    x[2, 7], y[3, 0] = float("inf"), float("nan")
    got = dg.int8_gemm(*(dg.int8_quantize(t.to(dev)) for t in (x, y)), out_dtype="f32")
    want = torch.zeros(M, N, dtype=torch.bool)
    want[2], want[:, 3] = True, True
    assert torch.equal(got.isnan().cpu(), want)


def test_product_without_columns_is_its_extras(dev):
    a = dg.int8_quantize(torch.empty(3, 0, device=dev))
    b = dg.int8_quantize(torch.empty(200, 0, device=dev))
    bias, src = torch.randn(200, device=dev), torch.randn(3, 200, device=dev)
    assert torch.equal(dg.int8_gemm(a, b, out_dtype="f32", bias_col=bias, source=src), bias + src)
    big = dg.int8_quantize(torch.empty(300, 0, device=dev))
    assert not bool(dg.int8_gemm(big, b).any())
    none = dg.int8_quantize(torch.empty(0, 64, device=dev))
    assert dg.int8_gemm(none, dg.int8_quantize(torch.ones(5, 64, device=dev))).shape == (0, 5)


@pytest.mark.parametrize("M,N,K", [(3, 100, 200), (50, 70, 300), (200, 300, 500), (4096, 4096, 200)])
def test_product_of_wider_storage(dev, M, N, K):
    """Operands that are views of larger ones: other rows and columns are not touched."""
    g = gen(14)
    a, b = operand(g, M, K, dev), operand(g, N, K, dev)
    want = dg.int8_gemm(a, b)
    width = a.data.shape[1]
    wide = []
    for q in (a, b):
        held = torch.full((q.data.shape[0] + 2, width + 48), 77, dtype=torch.int8, device=dev)
        held[1:-1, 16:16 + width] = q.data
        wide.append(dg.Int8Scaled(held[1:-1, 16:16 + width], q.scales, K))
    assert torch.equal(dg.int8_gemm(*wide), want)
    out = torch.full((M + 2, N), 3.0, dtype=BF16, device=dev)
    assert torch.equal(dg.int8_gemm(*wide, out=out[1:-1]), want)
    assert bool((out[0] == 3).all()) and bool((out[-1] == 3).all())


@pytest.mark.parametrize("M,N,K", [(20, 300, 500), (60, 500, 300), (1000, 2000, 1000), (2048, 2048, 700),
                                   (2000, 3000, 500), (3000, 2000, 500), (3000, 3000, 500), (4500, 2200, 400),
                                   (3000, 5000, 700), (1000, 1000, 20000), (700, 700, 30000),
                                   (700, 1000, 140000), (4096, 4096, 200)])
def test_product_of_rows_that_start_anywhere(dev, M, N, K):
    """Rows start at every multiple of 16 bytes from a line of memory on, in A and B alike or not; what
    lies before and behind them are the largest codes."""
    g = torch.Generator(device=dev).manual_seed(K)
    scales = [torch.rand(rows, generator=g, device=dev) + 0.5 for rows in (M, N)]
    data = [torch.randint(-127, 128, (rows, K), generator=g, device=dev, dtype=torch.int8) for rows in (M, N)]

    def held(i, start, pitch):
        rows, width = data[i].shape[0], R.up(K, 16) * 16
        flat = torch.full((start + rows * pitch + 64,), 127, dtype=torch.int8, device=dev)
        view = flat[start:].as_strided((rows, width), (pitch, 1))
        view[:, :K] = data[i]
        view[:, K:] = 0
        return dg.Int8Scaled(view, scales[i], K)

    even = R.up(K, 128) * 128
    want = dg.int8_gemm(held(0, 0, even), held(1, 0, even), out_dtype="f32")
    exact = torch.mm(data[0][:50].double(), data[1].double().t().contiguous())
    exact = exact * scales[0][:50].double()[:, None] * scales[1].double()
    R.within(want[:50], exact.cpu(), exact.cpu().abs() * 3 * U, "on lines")
    for start_a, more_a, start_b, more_b in ((0, 16, 0, 16), (16, 16, 112, 48), (96, 112, 32, 112), (64, 64, 0, 0),
                                             (0, 0, 48, 80), (112, 0, 112, 0), (80, 32, 16, 96)):
        got = dg.int8_gemm(held(0, start_a, even + more_a), held(1, start_b, even + more_b), out_dtype="f32")
        assert torch.equal(got, want), (start_a, more_a, start_b, more_b)


def test_product_overlaps_are_refused(dev):
    g = gen(15)
    a, b = operand(g, 40, 300, dev), operand(g, 24, 300, dev)
    held = randn(g, 41, 24).to(dev)
    before = held.clone()
    for kw in (dict(source=held[:40], out=held[1:]), dict(bias_col=held[3], out=held[:40])):
        with pytest.raises(ValueError, match="overlaps"):
            dg.int8_gemm(a, b, **kw)
    assert torch.equal(held, before)
    with pytest.raises(ValueError, match="overlaps"):
        one = operand(g, 24, 300, dev)
        dg.int8_gemm(a, dg.Int8Scaled(one.data, held.view(-1)[:24], 300), out=held[:40])
    assert torch.equal(dg.int8_gemm(a, b, source=held[1:], out=held[1:]),
                       dg.int8_gemm(a, b, out_dtype="f32", source=before[1:]))
    assert torch.equal(held[0], before[0])


def test_gradients_of_the_product(dev):
    """dA = dC B and dB = dC^T A in int8, against the formula on the codes' values: each operand is off by
    half a code of its row, s / 2."""
    g = gen(16)
    M, N, K = 200, 150, 333
    x, w, dc = (randn(g, *s) for s in ((M, K), (N, K), (M, N)))
    qx, qxt = dg.int8_quantize(x.to(dev), transposed="both")
    qw, qwt = dg.int8_quantize(w.to(dev), transposed="both")
    qd, qdt = dg.int8_quantize(dc.to(dev), transposed="both")
    x, w, dc = x.double(), w.double(), dc.double()

    def near(got, left, right, ql, qr):
        # sums of (l + dl)(r + dr) - l r with |dl| <= sl / 2, |dr| <= sr / 2, and the product's own rounding
        sl, sr = ql.scales.cpu().double()[:, None] / 2, qr.scales.cpu().double()[:, None] / 2
        n = left.shape[1]
        bound = sl * right.abs().sum(1) + left.abs().sum(1, keepdim=True) * sr.t() + n * sl * sr.t()
        R.within(got, left @ right.t(), bound * (1 + 2.0 ** -12), "gradient")

    near(dg.int8_gemm(qx, qw, out_dtype="f32"), x, w, qx, qw)
    near(dg.int8_gemm(qd, qwt, out_dtype="f32"), dc, w.t(), qd, qwt)
    near(dg.int8_gemm(qdt, qxt, out_dtype="f32"), dc.t(), x.t(), qdt, qxt)
    # against differences: the product is linear in A, so a step h along a code of A moves <C, dC> by h s dA
    h = 8
    a, b = qx, qw
    da = dg.int8_gemm(dg.int8_quantize(dc.to(dev).float()), qwt, out_dtype="f32").cpu().double()
    for i, k in ((0, 0), (7, 100), (199, 332)):
        moved = a.data.clone()
        code = int(moved[i, k])
        to = code + h if code < 100 else code - h
        moved[i, k] = to
        c0, c1 = (dg.int8_gemm(dg.Int8Scaled(d, a.scales, K), b, out_dtype="f32").double().cpu()
                  for d in (a.data, moved))
        slope = float(((c1 - c0) * dc).sum()) / ((to - code) * float(a.scales[i]))
        # dC and W^T are off by half a code each; C's elements by 3 U each, over the step
        s = float(qd.scales[i]) / 2, float(qwt.scales[k]) / 2
        bound = s[0] * float(w[:, k].abs().sum()) + s[1] * float(dc[i].abs().sum()) + N * s[0] * s[1]
        bound += float((6 * U * c0[i].abs() * dc[i].abs()).sum()) / (h * float(a.scales[i]))
        bound += float(qw.scales.max()) / 2 * float(dc[i].abs().sum())   # the product's own W
        assert abs(slope - float(da[i, k])) <= bound * 1.01, (slope, float(da[i, k]), bound)


# ---- graphs and streams -------------------------------------------------------------------------

def whole_layer(x, w, dy, bias):
    qx, qxt = dg.int8_quantize(x, transposed="both")
    qw, qwt = dg.int8_quantize(w, transposed="both")
    qd, qdt = dg.int8_quantize(dy, transposed="both")
    return [dg.int8_gemm(qx, qw, bias_col=bias), dg.int8_gemm(qd, qwt),
            dg.int8_gemm(qdt, qxt, out_dtype="f32"),
            dg.int8_gemm(dg.int8_quantize(x[:1]), qw, bias_col=bias)]


def layer_inputs(dev, seed):
    g = gen(seed)
    return [randn(g, 700, 4300).to(BF16).to(dev), randn(g, 520, 4300).to(dev),
            randn(g, 700, 520).to(BF16).to(dev), randn(g, 520).to(dev)]


def test_graph_replays_give_what_eager_calls_give(dev):
    held = layer_inputs(dev, 21)
    for _ in range(2):
        whole_layer(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = whole_layer(*held)
    for seed in (21, 22, 23):
        for t, n in zip(held, layer_inputs(dev, seed)):
            t.copy_(n)
        eager = [t.clone() for t in whole_layer(*held)]
        for t in outs:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (s, t) in enumerate(zip(outs, eager)):
            assert torch.equal(s, t), (seed, i)


def test_other_streams_give_the_same(dev):
    held = layer_inputs(dev, 24)
    want = whole_layer(*held)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            got.append(whole_layer(*held))
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        for i, (s, t) in enumerate(zip(outs, want)):
            assert torch.equal(s, t), (k, i)
