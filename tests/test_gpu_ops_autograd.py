"""What the operators write in place counts as changed for autograd; their results carry no history."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from test_gpu_ops import dev, gen, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def operands(dev):
    g = gen(61)
    return [dg.block_quantize(randn(g, n, 200).to(dev)) for n in (30, 20)]


def test_a_saved_tensor_that_is_written_is_refused(dev):
    a, b = operands(dev)
    w = torch.ones(20, device=dev, requires_grad=True)
    for write in (lambda t: dg.block_gemm(a, b, out=t),
                  lambda t: dg.block_gemm(a, b, source=t, out=t),
                  lambda t: dg.clip_grad_norm([t], 1e-3),
                  lambda t: dg.clip_grad_norm([t.clone()], 1e-3, out=[t]),
                  lambda t: dg.clip_grad_norm([torch.ones(7, device=dev), t[3:5]], 1e-3)):
        t = torch.ones(30, 20, device=dev)
        y = (t * w).sum()           # saves t
        at = t._version
        write(t)
        assert t._version == at + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


def test_what_is_only_read_is_as_it_was(dev):
    a, b = operands(dev)
    x = torch.ones(30, 20, device=dev)
    w = torch.ones(20, device=dev)
    o = torch.empty_like(x)
    _, mean, rstd = dg.layer_norm(x, w, w)
    dg.layer_norm_backward(x, x, w, mean, rstd)
    dg.block_gemm(a, b, bias_col=w, source=x)
    dg.grad_norm([x, w])
    dg.clip_grad_norm([x], 1.0, out=[o])
    dg.block_quantize(x)
    assert x._version == w._version == a.data._version == a.scales._version == mean._version == 0


def test_inference_tensors_are_written(dev):
    a, b = operands(dev)
    with torch.inference_mode():
        t = torch.zeros(30, 20, device=dev)
    dg.block_gemm(a, b, out=t)
    assert torch.equal(t, dg.block_gemm(a, b, out_dtype="f32"))
    dg.clip_grad_norm([t], 1e-3)
    assert abs(float(t.double().norm()) - 1e-3) < 1e-6


def test_results_carry_no_history(dev):
    x = torch.ones(30, 20, device=dev, requires_grad=True)
    w = torch.ones(20, device=dev, requires_grad=True)
    y, mean, rstd = dg.layer_norm(x, w)
    assert not any(t.requires_grad for t in (y, mean, rstd))
    assert not any(t.requires_grad for t in dg.layer_norm_backward(x, x, w, mean, rstd))
    assert not dg.grad_norm([x, w]).requires_grad
