"""Layer norm's backward pass where a row holds an infinity or a NaN."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
import ops_ref as R  # noqa: E402
from test_gpu_ops import BF16, F32, dev, gen, grad_bounds, norm_inputs, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(6, 300), (40, 1000), (700, 136), (600, 2500), (580, 9000), (30, 17000)])
@pytest.mark.parametrize("where", ["x", "dy"])
def test_layer_norm_backward_row_that_is_not_finite(dev, rows, cols, dtype, where):
    """Its own dx, and the sums over rows, have it; the other rows' dx do not."""
    print(f"layer norm backward {rows}x{cols} {dtype} inf in {where}", flush=True)
    g = gen(rows + cols)
    x, w, _ = norm_inputs(g, dev, rows, cols, dtype, F32)
    dy = randn(g, rows, cols).to(dtype).to(dev)
    row, col = rows - 2, cols // 2
    (x if where == "x" else dy)[row, col] = float("inf")
    _, mean, rstd = dg.layer_norm(x, w)
    dx, dw, db = dg.layer_norm_backward(dy, x, w, mean, rstd)
    assert not bool(torch.isfinite(dx[row]).any())
    keep = torch.arange(rows) != row
    args = [t[keep.to(dev)] for t in (dy, x)] + [w] + [t[keep.to(dev)] for t in (mean, rstd)]
    want, _, _ = R.norm_grad(*(t.cpu() for t in args))
    bound, _, _ = grad_bounds(args[0], args[1], *args[2:])
    R.within(dx[keep.to(dev)], want, bound + (want.abs() + bound) * R.HALF[dtype], "dx of the others")
    if where == "x":
        assert not bool(torch.isfinite(dw).any())
        total = dy.double().sum(0).cpu()
        slack = dy.double().abs().sum(0).cpu() * ((rows + 80) * R.U)
        R.within(db, total, slack + total.abs() * R.U, "db")
    else:
        odd = ~torch.isfinite(dw) | ~torch.isfinite(db)
        assert odd.nonzero().flatten().tolist() == [col]
