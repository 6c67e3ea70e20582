"""Outputs that overlap what other workgroups still read or write are refused by the public calls."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from test_gpu_ops import dev, gen, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_clip_of_a_gradient_that_is_there_twice(dev):
    g = randn(gen(51), 5000).to(dev)
    before = g.clone()
    with pytest.raises(ValueError, match="overlaps"):
        dg.clip_grad_norm([g, g], 1e-2)
    with pytest.raises(ValueError, match="overlaps"):
        dg.clip_grad_norm([g[:3000], g[2999:]], 1e-2)
    with pytest.raises(ValueError, match="overlaps"):
        dg.clip_grad_norm([g[:2000], g[2000:4000]], 1e-2, out=[g[2000:4000], g[:2000]])
    assert torch.equal(g, before)
    # read twice is no overlap
    one, two = torch.empty_like(g), torch.empty_like(g)
    norm = dg.clip_grad_norm([g, g], 1e-2, out=[one, two])
    assert torch.equal(one, two) and torch.equal(norm, dg.grad_norm([g, g]))
    assert abs(float(one.double().norm()) * 2 ** 0.5 - 1e-2) < 1e-5


def test_product_into_a_part_of_its_source(dev):
    g = gen(52)
    a, b = (dg.block_quantize(randn(g, n, 300).to(dev)) for n in (40, 24))
    held = randn(g, 41, 24).to(dev)
    before = held.clone()
    narrow = held.view(torch.bfloat16)[:20].view(40, 24)
    for kw in (dict(source=held[:40], out=held[1:]), dict(source=held[:40], out=narrow),
               dict(bias_col=held[3], out=held[:40])):
        with pytest.raises(ValueError, match="overlaps"):
            dg.block_gemm(a, b, **kw)
    assert torch.equal(held, before)
    want = dg.block_gemm(a, b, out_dtype="f32", source=before[1:])
    assert torch.equal(dg.block_gemm(a, b, source=held[1:], out=held[1:]), want)
    assert torch.equal(held[0], before[0])
