"""How the Python calls of the operators take their arguments (CPU: nothing here reaches a kernel)."""
import pytest

np = pytest.importorskip("numpy")
torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from dense_gemm_design_amd import ops as O  # noqa: E402


@pytest.mark.parametrize("transposed,sides", [(False, (True, False)), (True, (False, True)),
                                              ("both", (True, True)), (0, (True, False)),
                                              (1, (False, True)), (np.bool_(False), (True, False)),
                                              (np.bool_(True), (False, True))])
def test_quantise_takes_truth_values_of_any_type(monkeypatch, transposed, sides):
    """0, 1 and numpy's truth values ask for one side, as False and True do."""
    asked = []

    class Binding:
        @staticmethod
        def block_quantize(x, block, rows, cols, pow2):
            asked.append((rows, cols))
            return (x, x) * 2 if rows and cols else (x, x, None, None) if rows else (None, None, x, x)

    monkeypatch.setattr(O, "_binding", lambda: Binding)
    q = dg.block_quantize(torch.zeros(3, 5), transposed=transposed)
    assert asked == [sides] and all(type(s) is bool for s in asked[0])
    if sides == (True, True):
        assert isinstance(q, tuple) and (q[0].K, q[1].K) == (5, 3)
    else:
        assert isinstance(q, dg.BlockScaled) and q.K == (5 if sides[0] else 3)


@pytest.mark.parametrize("transposed", ["yes", "True", 2, None, (True,)])
def test_quantise_refuses_other_sides(transposed):
    with pytest.raises(ValueError, match="transposed must be"):
        dg.block_quantize(torch.zeros(3, 5), transposed=transposed)
