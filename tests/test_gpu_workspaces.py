"""Split-k workspaces on the GPU: graphs that leave them to the library beside
eager calls of the same stream.  A graph's products and the eager ones are
compared for equality with calls on workspaces of their own (split parts are
added in a fixed order, so the bits are the same)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g).to(BF16)


def test_fp8_graph_beside_eager_calls(dev):
    """The graph's FP8 product is the stream's first call with a workspace;
    then eager BF16 calls of the same stream, the backward pass with a larger
    workspace among them, between its replays."""
    fg8 = _fg8()
    g = torch.Generator().manual_seed(21)
    a, b = torch.randn(64, 2048, generator=g).to(dev), torch.randn(256, 2048, generator=g).to(dev)
    qa, sa = fg8.fp8_quantize(a, "1x128")
    qb, sb = fg8.fp8_quantize(b, "128x128")
    need = fg8.gemm_workspace_bytes(64, 256, 2048)
    assert need > 0
    x, w, dy = _bf16(g, 48, 2048).to(dev), _bf16(g, 200, 2048).to(dev), _bf16(g, 48, 200).to(dev)

    def own():
        return torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
    want_fp8 = fg8.gemm_fp8_blockscaled(qa, sa, qb, sb, workspace=own())
    want_y, want_z = fg8.gemm_bf16_epilogue(x, w, activation="silu", save_z=True, workspace=own())
    want_grads = fg8.gemm_bf16_epilogue_backward(dy, x, w, z=want_z, activation="silu", workspace=own())
    torch.cuda.synchronize()

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want_fp8)
    with torch.cuda.graph(graph, stream=stream):
        fg8.gemm_fp8_blockscaled(qa, sa, qb, sb, out=out)
    for i in range(4):
        with torch.cuda.stream(stream):
            y = fg8.gemm_bf16_epilogue(x, w, activation="silu")
            grads = fg8.gemm_bf16_epilogue_backward(dy, x, w, z=want_z, activation="silu")
            fp8 = fg8.gemm_fp8_blockscaled(qa, sa, qb, sb)
            big = [_bf16(g, 64, 4096 * (i + 1)).to(dev) for _ in range(2)]
            fg8.gemm_bf16_epilogue(*big)
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(fp8, want_fp8), f"eager {i}"
        assert all(torch.equal(p, q) for p, q in zip(grads, want_grads)), f"eager {i}"
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_fp8), f"replay {i}"
