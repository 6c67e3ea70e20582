"""An operator whose output finds no memory raises what torch raises."""
import pytest

torch = pytest.importorskip("torch")

import dense_gemm_design_amd as dg  # noqa: E402
from test_gpu_ops import dev  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_no_memory_is_torch_out_of_memory(dev):
    """With the allocator's limit put under what is in use (nothing is asked of the GPU)."""
    x = torch.ones(4096, 8192, device=dev)
    w = torch.ones(8192, device=dev)
    dg.layer_norm(x[:1], w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(dev).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (8 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            torch.empty_like(x)
        for call in (lambda: dg.layer_norm(x, w), lambda: dg.block_quantize(x),
                     lambda: dg.layer_norm_backward(x, x, w, x[:, 0].contiguous(), x[:, 0].contiguous())):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    y, _, _ = dg.layer_norm(x, w)
    assert not bool(y.any())
