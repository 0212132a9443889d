"""Memory that the loss's backward pass takes on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_frozen_head_takes_no_second_part(dev):
    """dx alone: the workspace of one part of the logits' gradients whatever dw's type
    would be, and the same dx as beside a float dw."""
    import moe_grouped_gemm_fp8_amd as fg8
    m, vocab, k = 2048, 20000, 256
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn(m, k, device=dev, generator=g).to(torch.bfloat16)
    w = (torch.randn(vocab, k, device=dev, generator=g) / 16).to(torch.bfloat16)
    t = torch.randint(0, vocab, (m,), device=dev, generator=g)
    _, lse = fg8.linear_cross_entropy(x, w, t)
    dloss = torch.full((m,), 1.0 / m, device=dev)
    size = fg8._lib.lib().fg8_linear_cross_entropy_backward_workspace_bytes
    one, two = (size(m, vocab, k, o) for o in (fg8._lib.OUT_BF16, fg8._lib.OUT_F32))
    assert two > one + 2 * m * vocab > fg8._lib.WS_KEEP_BYTES
    both = fg8.linear_cross_entropy_backward(dloss, x, w, t, lse)
    dx = None
    for dtype in (torch.float32, torch.bfloat16):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        dx, dw = fg8.linear_cross_entropy_backward(dloss, x, w, t, lse, dw_dtype=dtype, needs=(True, False))
        # (allocations are rounded up to 2 MB pieces at most)
        assert torch.cuda.max_memory_allocated() - before <= one + 2 * m * k + (4 << 20)
        assert dw is None and torch.equal(dx, both[0])
