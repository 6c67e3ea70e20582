"""Each kernel of the int8 product at shapes that go to it (test_int8_plan.py), against sums in 64 bits: every output
type, extra, alignment and size of scale.  The large tiles' workgroups go on to second and third tiles, and write
a tile beside the next one's first step."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from int8_shapes import TILES, WIDE, pitch  # noqa: E402
from test_gpu_ops import dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES, NAMES = [BF16, F32], ["bf16", "f32"]
U = R.U


@pytest.fixture(scope="module", autouse=True)
def large_tensors_go_back():
    """What torch keeps of them for other tests' tensors would count as memory in use there."""
    yield
    torch.cuda.empty_cache()


def operand(g, dev, rows, K, start):
    """Random codes between others: rows of `pitch`, from `start` bytes behind a line on where they may."""
    width, step = R.up(K, 16) * 16, pitch(K, start)
    held = torch.full(((rows + 1) * step + 256,), 127, dtype=torch.int8, device=dev)
    first = 128 if start % 128 == 0 else 128 + start
    view = held[first:].as_strided((rows, width), (step, 1))
    view[:, :K] = torch.randint(-127, 128, (rows, K), generator=g, device=dev, dtype=torch.int8)
    view[:, K:] = 0
    scales = torch.exp(torch.randn(rows, generator=g, device=dev)) * 1e-2
    return dg.Int8Scaled(view, scales, K)


def exact_sums(a, b):
    return torch.mm(a.values.double(), b.values.double().t().contiguous())


def near(got, sums, a, b, out, what, bias=None, source=None):
    """got against the formula in 64 bits: the sum's rounding, its product with one scale, the next product with the
    bias added, the source added, and the output's own."""
    t = sums * a.scales.double()[:, None] * b.scales.double()
    z = t if bias is None else t + bias.double()
    want = z if source is None else z + source.double()
    bound = 2 * U * t.abs() + U * z.abs() + R.HALF[out] * want.abs() * (1 + 4 * U) + 2.0 ** -148
    if source is not None:
        bound += U * want.abs()
    bad = ~((got.double() - want).abs() <= bound * (1 + 2.0 ** -20))
    assert got.dtype == out
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} outside, first at {i}: {float(got[i])} for "
                             f"{float(want[i])} +- {float(bound[i])}")


def run(a, b, kind, **kw):
    return dg.int8_gemm(a, b, out_dtype="bf16" if kind == BF16 else "f32", **kw)


def guarded(M, N, out, dev, by):
    """A tensor for C that starts `by` elements behind a multiple of 16 bytes, between others that stay."""
    flat = torch.full((M * N + 64,), 3.0, dtype=out, device=dev)
    return flat, flat[16 + by:16 + by + M * N].view(M, N)


def untouched(flat, by, n):
    return bool((flat[:16 + by] == 3).all()) and bool((flat[16 + by + n:] == 3).all())


@pytest.mark.parametrize("out", TYPES, ids=NAMES)
@pytest.mark.parametrize("M,N,K,start,kernel", WIDE + TILES)
def test_extras_and_alignments(dev, M, N, K, start, kernel, out):
    print(f"int8 {kernel}: {M}x{N}x{K} rows at {start} {out}", flush=True)
    g = torch.Generator(device=dev).manual_seed(M + N + K)
    a, b = operand(g, dev, M, K, start), operand(g, dev, N, K, start)
    sums = exact_sums(a, b)
    randn = lambda *s: torch.randn(*s, generator=g, device=dev) * 30   # noqa: E731
    bias, sources = randn(N), [randn(M, N), randn(M, N).to(BF16)]
    near(run(a, b, out), sums, a, b, out, "plain")
    for by in (0, 1):
        flat, c = guarded(M, N, out, dev, by)
        run(a, b, out, bias_col=bias, out=c)
        near(c, sums, a, b, out, f"bias, {by} off", bias)
        assert untouched(flat, by, M * N), f"behind C, {by} off"
    for source in sources:
        for vector in (None, bias):
            near(run(a, b, out, bias_col=vector, source=source), sums, a, b, out, f"source {source.dtype}", vector,
                 source)
        if source.dtype != out:
            continue
        for by in (0, 1):
            flat, c = guarded(M, N, out, dev, by)
            c.copy_(source)
            run(a, b, out, bias_col=bias, source=c, out=c)
            near(c, sums, a, b, out, f"in place, {by} off", bias, source)
            assert untouched(flat, by, M * N), f"behind C in place, {by} off"


@pytest.mark.parametrize("out", TYPES, ids=NAMES)
@pytest.mark.parametrize("M,N,K,start,kernel", WIDE + TILES)
def test_scales_of_any_size_and_rows_that_are_no_numbers(dev, M, N, K, start, kernel, out):
    print(f"int8 scales {kernel}: {M}x{N}x{K} rows at {start} {out}", flush=True)
    g = torch.Generator(device=dev).manual_seed(M + N + K + 1)
    a, b = operand(g, dev, M, K, start), operand(g, dev, N, K, start)
    sums = exact_sums(a, b)
    fine = a.scales.clone()
    # all of A's over 2^90; in one row of 300 only; under fp32's smallest normal number beside large ones
    for few, ea, eb in ((False, 110, -115), (True, 100, -90), (False, -130, 115)):
        a.scales.copy_(fine)
        rows = slice(None, None, 300) if few else slice(None)
        a.scales[rows] = 2.0 ** ea
        b.scales.copy_((1 + torch.rand(N, generator=g, device=dev)) * 2.0 ** eb)
        near(run(a, b, out), sums, a, b, out, f"scales of 2^{ea} and 2^{eb}")
    a.scales.copy_(fine)
    b.scales.copy_(torch.rand(N, generator=g, device=dev) + 0.5)
    odd_m, odd_n = [0, M // 2, M - 1], [1, N // 2, N - 1]
    a.scales[odd_m] = float("nan")
    b.scales[odd_n] = float("nan")
    got = run(a, b, out)
    nan = torch.zeros(M, N, dtype=torch.bool, device=dev)
    nan[odd_m] = True
    nan[:, odd_n] = True
    assert torch.equal(got.isnan(), nan)


@pytest.mark.parametrize("M,N,K,start,kernel", WIDE + TILES)
def test_rows_have_the_same_bits_alone(dev, M, N, K, start, kernel):
    """The first rows, the last one and those around the tiles' edges."""
    g = torch.Generator(device=dev).manual_seed(M + N + K + 2)
    a, b = operand(g, dev, M, K, start), operand(g, dev, N, K, start)
    source = torch.randn(M, N, generator=g, device=dev)
    for out in TYPES:
        for kw in ({}, dict(source=source)):
            whole = run(a, b, out, **kw)
            for m in {0, 1, 63, 64, 127, 128, 191, 192, 255, 256, 511, 512, M - 1}:
                if m < M:
                    one = dg.Int8Scaled(a.data[m:m + 1], a.scales[m:m + 1], K)
                    alone = run(one, b, out, **{k: v[m:m + 1] for k, v in kw.items()})
                    assert torch.equal(alone[0], whole[m]), (out, m)


def test_large_tiles_at_once_on_two_streams(dev):
    """Two products of many rounds beside each other, each into its own tensor."""
    g = torch.Generator(device=dev).manual_seed(9)
    M, N, K, start, _ = WIDE[2]
    pairs = [(operand(g, dev, M, K, start), operand(g, dev, N, K, start)) for _ in range(2)]
    want = [run(*p, F32) for p in pairs]
    torch.cuda.synchronize()
    got = []
    for p, s in zip(pairs, (torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(s):
            got.append([run(*p, F32) for _ in range(3)])
    torch.cuda.synchronize()
    for w, cs in zip(want, got):
        for c in cs:
            assert torch.equal(c, w)
