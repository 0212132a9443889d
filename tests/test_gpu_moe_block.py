"""examples/moe_block.py, forward and backward, against torch's autograd in
float64 on the CPU.

Both sides take the same BF16 parameters and input and the same routing (the
GPU's).  The GPU rounds to BF16 at eight places in a row at most between an
input and a gradient, each by up to 2^-8 and 2^-9.3 rms, and the steps pass a
relative error on with a gain near one: 8 * 2^-9.3 = 0.013 rms if all added up;
twice that, 0.026, bounds the relative 2-norm of every output.  Where relu's
input changes sign under such an error the gradient's term flips whole: the
share of elements within 2^-8 of zero is about 0.003, whose norm is 0.055 of
the whole; gradients behind relu get 0.08.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [(1, 128, 64, 4, 1), (77, 256, 192, 8, 2), (300, 384, 256, 6, 3)])
def test_block_against_autograd(dev, tokens, hidden, inter, experts, topk):
    print(f"moe block {tokens} tokens {hidden}x{inter}, {experts} experts, top {topk}", flush=True)
    block = _example().MoeBlock(hidden, inter, experts, topk, device=dev)
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    dout = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    out, saved = block.forward(x.to(dev))
    dx, grads = block.backward(dout.to(dev), saved)
    ids = saved[4].cpu()

    names = ["norm_w", "norm_b", "wr", "br", "ws1", "bs1", "ws2", "bs2", "w1", "w2"]
    v = {n: getattr(block, n).cpu().double().requires_grad_() for n in names}
    t = x.double().requires_grad_()
    h = torch.nn.functional.layer_norm(t, (hidden,), v["norm_w"], v["norm_b"])
    p = torch.softmax((h @ v["wr"].T + v["br"]).gather(1, ids), 1)
    s = torch.nn.functional.gelu(h @ v["ws1"].T + v["bs1"]) @ v["ws2"].T + v["bs2"] + t
    routed = torch.zeros_like(s)
    for j in range(topk):
        w1, w2 = v["w1"][ids[:, j]], v["w2"][ids[:, j]]
        a = torch.relu((w1 @ h[:, :, None])[:, :, 0])
        routed = routed + p[:, j:j + 1] * (w2 @ a[:, :, None])[:, :, 0]
    want = s + routed
    want.backward(dout.double())

    def close(got, ref, bound, what):
        off = float((got.cpu().double() - ref).norm() / ref.norm())
        assert off <= bound, f"{what}: relative error {off:.4f} over {bound}"

    close(out, want.detach(), 0.026, "out")
    close(dx, t.grad, 0.08, "dx")
    for n in names:
        if n in ("wr", "br") and topk == 1:      # a softmax over one logit has no gradient
            assert not grads[n].any()
        else:
            close(grads[n], v[n].grad, 0.026 if n in ("ws2", "bs2", "w2") else 0.08, n)
