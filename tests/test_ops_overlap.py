"""Outputs that overlap what other workgroups still read or write are refused (C ABI, on the CPU: every call
here returns before anything is enqueued)."""
import ctypes
import random

import pytest

torch = pytest.importorskip("torch")

from dense_gemm_design_amd import _lib as L  # noqa: E402
from dense_gemm_design_amd import ops as O  # noqa: E402

P = 1 << 20


def clip(entries):
    """Status of a clipping call without a workspace, so that a list that is in order gets no further."""
    arr = (O.GemmTensor * len(entries))(*[O.GemmTensor(*e) for e in entries])
    return O.load().gemm_clip_grad_norm(arr, len(entries), 1.0, P, None, 0, None)


def test_clip_refuses_what_overlaps():
    inv, ok = L.GEMM_ERR_INVALID_ARG, L.GEMM_ERR_WORKSPACE
    f32, bf16 = L.GEMM_F32, L.GEMM_BF16
    g, h, o, q = P, P + (1 << 16), P + (2 << 16), P + (3 << 16)
    n = 100
    for entries, want in (
            ([(g, g, n, f32), (h, h, n, f32)], ok),
            ([(h, h, n, f32), (g, g, n, f32)], ok),
            ([(g, g, n, f32), (g, g, n, f32)], inv),                  # twice, in place
            ([(g, o, n, f32), (g, q, n, f32)], ok),                   # twice, out of place
            ([(g, o, n, f32), (h, o, n, f32)], inv),                  # one output for two
            ([(g, h, n, f32), (h, g, n, f32)], inv),                  # outputs exchanged
            ([(g, g + 16, n, f32)], inv),                             # shifted over its own data
            ([(g, g - 16, n, f32)], inv),
            ([(g, g, n, f32), (g + 4 * n, g + 4 * n, n, f32)], ok),   # neighbours
            ([(g, g, n, f32), (g + 4 * n - 2, g + 4 * n - 2, n, bf16)], inv),
            ([(g, g, n, bf16), (g + 2 * n, g + 2 * n, n, bf16)], ok),
            ([(g, g, n, f32), (g + 40, o, 3, f32)], inv),             # inside what is scaled in place
            ([(g, g, n, f32), (g + 40, g + 40, 0, f32)], ok),         # of nothing
            ([(g, o, n, f32), (g + 40, q, 3, f32)], ok)):             # inside what is only read
        assert clip(entries) == want, entries


@pytest.mark.parametrize("into", [False, True], ids=["in_place", "into"])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed", "two buffers"])
def test_clip_finds_an_overlap_in_long_lists(order, into):
    rng = random.Random(len(order))
    sizes = [rng.randint(1, 3000) for _ in range(300)]
    at, entries, far = P, [], 1 << 36
    for k, n in enumerate(sizes):
        t = L.GEMM_F32 if k % 3 else L.GEMM_BF16
        base = at if order != "two buffers" or t == L.GEMM_F32 else at + (1 << 34)
        entries.append((base, base + far if into else base, n, t))
        at = (at + n * (4 if t == L.GEMM_F32 else 2) + 3) // 4 * 4 + rng.choice([0, 256])
    if order == "falling":
        entries.reverse()
    if order == "mixed":
        rng.shuffle(entries)
    assert clip(entries) == L.GEMM_ERR_WORKSPACE
    for _ in range(20):
        i, j = rng.sample(range(300), 2)
        bad = list(entries)
        d, o, n, t = bad[i]
        es = 4 if t == L.GEMM_F32 else 2
        other = bad[j]
        width = other[2] * (4 if other[3] == L.GEMM_F32 else 2)
        # i's output begins within, or ends within, what is written for j
        begin = other[1] + (rng.randrange(0, width, 4) if rng.random() < 0.5 else -rng.randrange(0, n * es, 4))
        bad[i] = (d if into else begin, begin, n, t)
        if begin + n * es > other[1]:
            assert clip(bad) == L.GEMM_ERR_INVALID_ARG, (i, j)


def back(dx, dy, dstride, x, stride, rows=5, cols=64, dtype=L.GEMM_F32):
    """Status of a norm's backward pass without a workspace."""
    w = P << 8
    return O.load().gemm_layer_norm_backward(dy, dstride, x, stride, dtype, rows, cols, w, L.GEMM_F32, w, w,
                                             dx, w, w, None, 0, None)


def test_norm_backward_refuses_a_dx_over_rows_of_another_stride():
    inv, ok = L.GEMM_ERR_INVALID_ARG, L.GEMM_ERR_WORKSPACE
    x, dy = P, P + (1 << 20)
    row = 64 * 4
    for args, want in (((dy + (1 << 20), dy, 64, x, 64), ok),
                       ((x, dy, 64, x, 64), ok), ((dy, dy, 64, x, 64), ok),      # each row over its own
                       ((x, dy, 64, x, 65), inv), ((x, dy, 64, x, 128), inv),
                       ((dy, dy, 65, x, 64), inv), ((dy, dy, 0, x, 64), inv),    # one row for all
                       ((x, dy, 64, x, 0), inv),
                       ((x + row, dy, 64, x, 64), inv), ((x - row, dy, 64, x, 64), inv),
                       ((x + 5 * row, dy, 64, x, 64), ok), ((x - 5 * row, dy, 64, x, 64), ok),
                       ((x + 5 * row - 4, dy, 64, x, 64), inv), ((x - 5 * row + 4, dy, 64, x, 64), inv),
                       ((x + row, dy, 64, x, 64 * 6), ok),                        # between two rows
                       ((x + row, dy, 64, x, 64 * 6 - 1), inv),
                       ((x + 2 * 6 * row + row, dy, 64, x, 64 * 6), ok),
                       ((x + 2 * 6 * row + row - 4, dy, 64, x, 64 * 6), inv),
                       ((x + 4 * 6 * row + row, dy, 64, x, 64 * 6), ok),          # behind the last
                       ((dy, dy, 0, x, 64, 1), ok), ((x, dy, 64, x, 99, 1), ok)):  # one row: no stride
        assert back(*args) == want, args


def test_norm_backward_overlaps_against_plain_sets():
    rng = random.Random(3)
    far = P << 4
    for _ in range(3000):
        rows, cols = rng.randint(1, 5), rng.randint(1, 6)
        stride = rng.choice([0, cols, cols + rng.randint(1, 40)])
        at = rng.randint(-60, 200)
        own = {e for r in range(rows) for e in range(r * stride, r * stride + cols)}
        out = set(range(at, at + rows * cols))
        want = not (own & out) or (at == 0 and (rows == 1 or stride == cols))
        for dtype, es in ((L.GEMM_F32, 4), (L.GEMM_BF16, 2)):
            got = back(P + at * es, far, cols, P, stride, rows, cols, dtype)
            assert got == (L.GEMM_ERR_WORKSPACE if want else L.GEMM_ERR_INVALID_ARG), (rows, cols, stride, at)
            got = back(P + at * es, P, stride, far, cols, rows, cols, dtype)
            assert got == (L.GEMM_ERR_WORKSPACE if want else L.GEMM_ERR_INVALID_ARG), (rows, cols, stride, at)


def product(C, source=None, bias=None, M=100, N=90, dtype_c=L.GEMM_F32, dtype_source=L.GEMM_F32):
    """Status of a product that needs a workspace and has none."""
    far = P << 8
    d = O.GemmBlockDesc(M=M, N=N, K=9000, lda=9008, ldb=9008, scale_lda=M, scale_ldb=N, dtype_c=dtype_c,
                        dtype_source=dtype_source)
    return O.load().gemm_block_run(d, far, far, far, far, C, bias, source, None, 0, None)


def test_product_refuses_a_source_or_bias_that_overlaps_c():
    inv, ok, bf16 = L.GEMM_ERR_INVALID_ARG, L.GEMM_ERR_WORKSPACE, L.GEMM_BF16
    all_f32 = 100 * 90 * 4
    for kw, want in ((dict(source=P), ok), (dict(source=P, dtype_c=bf16, dtype_source=bf16), ok),
                     (dict(source=P, dtype_c=bf16), inv), (dict(source=P, dtype_source=bf16), inv),
                     (dict(source=P + 4), inv), (dict(source=P - 360), inv),
                     (dict(source=P + all_f32), ok), (dict(source=P - all_f32), ok),
                     (dict(source=P + all_f32 - 4), inv), (dict(source=P - all_f32 + 4), inv),
                     (dict(source=P + all_f32 // 2, dtype_c=bf16), ok),
                     (dict(source=P - all_f32 // 2, dtype_source=bf16), ok),
                     (dict(bias=P), inv), (dict(bias=P + 400), inv), (dict(bias=P - 360), ok),
                     (dict(bias=P - 356), inv), (dict(bias=P + all_f32), ok),
                     (dict(bias=P, M=1), ok), (dict(bias=P, M=1, dtype_c=bf16), inv)):
        assert product(P, **kw) == want, kw
