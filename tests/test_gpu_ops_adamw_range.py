"""The AdamW step where its numbers are at the ends of their range."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from test_gpu_ops import dev, gen, randn  # noqa: E402,F401
from test_gpu_ops_adamw import KEYS, step_and_check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state", ["e4m3", "f32"])
@pytest.mark.parametrize("eps", [2.0 ** -100, 2.0 ** -101, 2.0 ** -126, 1e-38, 1e-40, 1e-45, 1e-300])
def test_eps_of_any_size(dev, eps, state):
    """Moments of zero over any eps are zero, and small ones what the formula says, whether or not eps and
    the quotient's other side are normal numbers."""
    g = gen(20)
    params = [randn(g, 700).to(dev)]
    before = params[0].clone()
    for step in (1, torch.tensor(2, device=dev)):
        zeros = [torch.zeros(700, device=dev)]
        dg.adamw_step(params, zeros, dg.adamw_state(params, state), step, **{**KEYS, "eps": eps, "weight_decay": 0.0})
        assert torch.equal(params[0], before)
        grads = [randn(g, 700).to(dev) * 1e-3]
        grads[0][::3] = 0
        step_and_check(params, grads, dg.adamw_state(params, state), step, f"eps {eps}", eps=eps)
        before = params[0].clone()
    if state == "f32" and 1e-45 < eps < 2.0 ** -100:
        # a first moment of some 2^-20 times the rate's reciprocal and eps over a second one of zero: no
        # smaller than 2^-125, where fp32 has all its places
        s = dg.adamw_state(params, state)
        s.m[:700] = max(eps * 1e4, 2.0 ** -125)
        step_and_check(params, [torch.zeros(700, device=dev)], s, 3, f"eps {eps} alone", eps=eps)


def test_scales_are_the_rounded_quotient(dev):
    """Where moments are the gradients (no memory), a block's scale is amax / 448 rounded to nearest.  (The
    exact quotient is no fp32 midpoint, and further from one than fp64's places: it is one of sevenths.)"""
    g = gen(21)
    n = 4000 * 128
    x = randn(g, n) * torch.exp(randn(g, 4000) * 8).repeat_interleave(128)
    p = torch.zeros(n, device=dev)
    s = dg.adamw_state([p], "e4m3")
    dg.adamw_step([p], [x.to(dev)], s, 1, 1e-3, betas=(0.0, 0.0))
    want = (x.view(-1, 128).abs().amax(1).double() / 448).float()
    assert float(want.min()) > 2.0 ** -126
    assert torch.equal(s.m_scales.cpu(), want)
