"""A bf16 C with exact=True keeps 24 places of every sum, on tiles of every number of rows."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from test_gpu_ops import BF16, dev, fp32_bound, gen, operand, randn  # noqa: E402,F401
from test_gpu_ops_scales import KINDS, kinds  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def cancelling(g, dev, M, N, K, block, pow2):
    """Operands of which each eight k have two large products that are each other's opposite, and six that
    are 2^-14 of their size and positive: what the sum is made of."""
    a, b = torch.full((M, K), 2.0), torch.full((N, K), 2.0)
    for t, rows, sign in ((a, M, -1), (b, N, 1)):
        large = 256 * torch.randn(rows, R.up(K, 8), generator=g).sign()
        t[:, 0::8] = large
        t[:, 1::8] = sign * large[:, :t[:, 1::8].shape[1]]
    if K % 8 == 1:                       # one that has no partner
        a[:, -1] = 0
    return [(dg.block_quantize(t.to(dev), kind, pow2=pow2)) for t, kind in ((a, "row"), (b, block))]


@kinds
@pytest.mark.parametrize("M,N,K", [(33, 200, 384), (300, 390, 1000), (140, 139, 5001), (4096, 4352, 384),
                                   (4096, 4096, 256)])
def test_cancelling_terms_keep_their_small_ones(dev, M, N, K, block, pow2):
    print(f"exact {M}x{N}x{K} b {block} pow2={pow2}", flush=True)
    a, b = cancelling(gen(M + N + K), dev, M, N, K, block, pow2)
    av = R.spread(a.data, a.scales, "row", K).to(dev)
    bv = R.spread(b.data, b.scales, block, K).to(dev)
    want = torch.mm(av, bv.t().contiguous())
    size = torch.mm(av.abs(), bv.abs().t().contiguous())
    # six products of 4 in eight, beside two of 2^16: an error of 24 against a bound of about 2^17 300 2^-24 = 2.3
    bound = fp32_bound(size, K)
    got = dg.block_gemm(a, b, exact=True)
    assert got.dtype is BF16
    bad = ~((got.double() - want).abs() <= bound + (want.abs() + bound) * R.HALF[BF16])
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())
    # the same numbers as an fp32 C, rounded
    assert torch.equal(got, dg.block_gemm(a, b, out_dtype="f32").to(BF16))


@kinds
@pytest.mark.parametrize("M,N,K", [(5, 100, 300), (100, 250, 1100), (1000, 3, 200), (2171, 2045, 4300),
                                   (4099, 4201, 130)])
def test_exact_with_extras(dev, M, N, K, block, pow2):
    g = gen(M + N + K)
    a, av = operand(g, dev, M, K, "row", pow2)
    b, bv = operand(g, dev, N, K, block, pow2)
    bias, src = randn(g, N).to(dev), randn(g, M, N).to(BF16).to(dev)
    want = torch.mm(av.to(dev), bv.to(dev).t().contiguous()) + bias.double() + src.double()
    bound = fp32_bound(torch.mm(av.to(dev).abs(), bv.to(dev).abs().t().contiguous()), K)
    bound = bound + (bias.double().abs() + src.double().abs()) * (2 * R.U)
    whole = torch.full((M + 2, N), 7.0, dtype=BF16, device=dev)
    dg.block_gemm(a, b, bias_col=bias, source=src, out=whole[1:-1], exact=True)
    bad = ~((whole[1:-1].double() - want).abs() <= bound + (want.abs() + bound) * R.HALF[BF16])
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist())
    assert bool((whole[0] == 7).all()) and bool((whole[-1] == 7).all())
