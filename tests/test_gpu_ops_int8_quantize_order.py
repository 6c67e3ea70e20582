"""int8 quantisation of over 2048 rows whose workgroups take the blocks of columns in another order than they lie
in (columns in multiples of eight parts of two, four or six blocks of 128): every block is written, by its own
scales."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_ops import dev, gen, randn  # noqa: E402,F401
from test_gpu_ops_int8 import NAMES, TYPES, check_quantize  # noqa: E402

pytestmark = pytest.mark.gpu


def parts_and_order(cols):
    """Blocks of 128 columns, how many of them a part has, and the order that their workgroups come in."""
    blocks = -(-cols // 128)
    wide = -(-blocks // 16)
    if blocks % (8 * wide):
        return blocks, wide, list(range(blocks))
    return blocks, wide, [((b // 8) // wide * 8 + b % 8) * wide + (b // 8) % wide for b in range(blocks)]


SHAPES = [(2060, 4000), (2100, 4096), (2049, 8070), (2049, 12285)]


@pytest.mark.parametrize("dtype", TYPES, ids=NAMES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_blocks_in_another_order(dev, rows, cols, dtype):
    blocks, wide, order = parts_and_order(cols)
    assert wide >= 2 and order != list(range(blocks)) and sorted(order) == list(range(blocks))
    print(f"int8 quantize {rows}x{cols} {dtype}", flush=True)
    g = gen(rows + cols)
    x = randn(g, rows, cols) * torch.exp(randn(g, rows, 1) * 3) * torch.exp(randn(g, 1, cols))
    x = x.to(dtype).to(dev)
    for side in (False, True, "both"):
        check_quantize(x, side, f"{rows}x{cols} side {side}")
