"""Which second moments an e4m3 state of the AdamW step follows."""
import warnings

import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from test_gpu_ops import dev, gen, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("state,betas", [("e4m3", (0.9, 0.95)), ("f32", (0.9, 0.999))])
def test_betas_that_are_not_given(dev, state, betas):
    g = gen(30)
    p = [randn(g, 1000).to(dev)]
    q, s, t = [p[0].clone()], dg.adamw_state(p, state), dg.adamw_state(p, state)
    for k in (1, 2, 3):
        d = [randn(g, 1000).to(dev)]
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            dg.adamw_step(p, d, s, k, 1e-2)
            dg.adamw_step(q, d, t, k, 1e-2, betas=betas)
    assert torch.equal(p[0], q[0])
    for a, b in zip(s.moments(), t.moments()):
        assert torch.equal(a, b)


def test_a_beta2_that_e4m3_does_not_follow(dev):
    p, d = [torch.zeros(300, device=dev)], [torch.ones(300, device=dev)]
    with pytest.warns(UserWarning, match="beta2 of 0.999"):
        dg.adamw_step(p, d, dg.adamw_state(p, "e4m3"), 1, 1e-3, betas=(0.9, 0.999))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        dg.adamw_step(p, d, dg.adamw_state(p, "f32"), 1, 1e-3, betas=(0.9, 0.999))
        with pytest.raises(ValueError, match="beta2 must be a finite number"):
            dg.adamw_step(p, d, dg.adamw_state(p, "e4m3"), 1, 1e-3, betas=(0.9, float("-inf")))


@pytest.mark.parametrize("fall", [1 / 3, 0.1, 0.01])
def test_second_moments_follow_their_gradients(dev, fall):
    """With the betas that are not given: of each 128, 120 have gradients that fall to a share of the others'.
    The step's own rounding leaves a root within one code, an eighth, of the one that fp32 holds for as many of
    them above it as below."""
    g = torch.Generator(device=dev).manual_seed(31)
    n = 64 * 128
    p, s = [torch.zeros(n, device=dev)], None
    s = dg.adamw_state(p, "e4m3")
    small = torch.arange(n, device=dev) % 128 >= 8
    v = torch.zeros(n, dtype=torch.float64, device=dev)
    for t in range(1, 801):
        d = torch.randn(n, generator=g, device=dev)
        if t > 400:   # 0.95^200 of what was is left in the middle of the rest, 10^-9 of v at its end
            d = torch.where(small, d * fall, d)
        dg.adamw_step(p, [d], s, t, 1e-3)
        v = 0.95 * v + 0.05 * d.double().square()
    ratio = (s.moments()[1].double() / v).sqrt()[small]
    assert 8 / 9 < float(ratio.median()) < 9 / 8, float(ratio.median())
    assert 0.5 < float(ratio.min()) and float(ratio.max()) < 2, (float(ratio.min()), float(ratio.max()))
