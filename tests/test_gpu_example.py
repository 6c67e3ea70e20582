"""The example of the operators around the product, at small sizes."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("pow2", [False, True], ids=["any", "pow2"])
def test_fp8_linear_learns(pow2):
    """The loss falls by more than half in 30 steps, and a token alone gets what it gets in a batch."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_linear
    losses, layer = fp8_linear.train(700, 300, 200, steps=30, pow2=pow2, say=None)
    assert all(b == b for b in losses) and losses[-1] < 0.5 * losses[0], losses
    x = torch.randn(40, 300, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x = x.to(torch.bfloat16)
    batch, alone = layer.forward(x), torch.cat([layer.token(x[i:i + 1]) for i in range(4)])
    # the same codes and scales: both differ from the exact sum by the bf16 rounding of y (2^-8) and
    # by the batch's alignment of products, under 2^-9 of sqrt(K) terms' size here
    assert bool(((batch[:4].float() - alone.float()).abs() <=
                 2 * 2.0 ** -8 * alone.float().abs() + 2.0 ** -9 * 300 ** 0.5).all())


def test_fp8_linear_gradients_are_near_the_fp32_ones():
    """Codes are off by 2^-4 relative, so a product of two by 2^-3 of a term; over the sums of hundreds
    of independent terms the gradients' 2-norm is off by less than that."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_linear
    layer = fp8_linear.NormLinear(260, 390, "cuda")
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(500, 260, device="cuda", generator=g).to(torch.bfloat16)
    dy = torch.randn(500, 390, device="cuda", generator=g).to(torch.bfloat16)
    layer.forward(x)
    grads, dx = layer.backward(dy)
    leaves = [p.detach().clone().requires_grad_() for p in (x.float(), *layer.parameters)]
    X, gain, shift, w, b = leaves
    h = torch.nn.functional.layer_norm(X, (260,), gain, shift)
    (h.matmul(w.t()) + b).backward(dy.float())
    for got, leaf in zip([dx, *grads], leaves):
        want = leaf.grad
        assert float((got.float() - want).norm() / want.norm()) < 2.0 ** -3
