"""The operators as a training step runs them: routed gated experts, the way back to
the tokens onto the residual stream, the loss of a linear head, and the gradients of
everything, against torch's autograd in float64 on the CPU with the same BF16
parameters and routing.

The GPU rounds to BF16 at nine places in a row at most between a parameter and its
gradient (z, h, y, the stream; dlogits, the stream's gradient, dy, dh, dz), each by up
to 2^-8 and 2^-9.3 rms; the steps pass a relative error on with a gain near one:
9 * 2^-9.3 = 0.0143 rms if all added up; twice that, 0.029, bounds the relative 2-norm
of every output.  The loss takes the stream's rounding only: its rows' logits are off by
2^-9.3 of their length, 3.5 here, and a row's loss by twice that at most: 0.012 rms.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk,vocab", [(1, 128, 64, 4, 1, 50), (77, 256, 104, 8, 2, 1003),
                                                                    (300, 384, 264, 6, 3, 4096)])
def test_step_against_autograd(dev, tokens, hidden, inter, experts, topk, vocab):
    import moe_grouped_gemm_fp8_amd as fg8
    print(f"step {tokens} tokens {hidden}x{inter}, {experts} experts, top {topk}, {vocab} classes", flush=True)
    g = torch.Generator().manual_seed(tokens)

    def weight(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale * shape[-1] ** -0.5).to(BF16)
    x = torch.randn(tokens, hidden, generator=g).to(BF16)
    w1, w2, head = weight(experts, 2 * inter, hidden, scale=2.0), weight(experts, hidden, inter), weight(vocab, hidden, scale=2.0)
    ids = torch.stack([torch.randperm(experts, generator=g)[:topk] for _ in range(tokens)])
    p = torch.softmax(torch.randn(tokens, topk, generator=g), 1)
    target = torch.randint(0, vocab, (tokens,), generator=g)
    if tokens > 4:
        target[::4] = -100
    live = target >= 0
    count = int(live.sum())

    # the step
    X, W1, W2, H = x.to(dev), w1.to(dev), w2.to(dev), head.to(dev)
    lay = fg8.moe_contiguous_layout_fp8(X, ids.to(torch.int32).to(dev), experts)
    off, token = lay["expert_offsets"], lay["row_token"].long()
    rows = torch.where((token >= 0)[:, None], X[token.clamp(min=0)], 0)
    h, z = fg8.grouped_gemm_bf16_gated(rows, W1, off, save_z=True)
    y = fg8.grouped_gemm_bf16(h, W2, off)
    s = fg8.moe_combine(y, lay["token_row"], p.to(dev), residual=X)
    loss, lse = fg8.linear_cross_entropy(s, H, target.to(dev))
    ds, dhead = fg8.linear_cross_entropy_backward(torch.full((tokens,), 1.0 / count, device=dev), s, H, target.to(dev), lse)
    dy, dp = fg8.moe_combine_backward(ds, y, lay["token_row"], lay["row_token"], p.to(dev))
    dw2 = fg8.grouped_gemm_bf16_wgrad(dy, h, off)
    dh = fg8.grouped_gemm_bf16_dgrad(dy, W2, off)
    drows, dw1 = fg8.grouped_gemm_bf16_gated_backward(dh, rows, W1, z, off)
    dx = fg8.moe_combine(drows, lay["token_row"], torch.ones(tokens, topk, device=dev), residual=ds)

    # the same by autograd
    v = {n: t.double().requires_grad_() for n, t in (("x", x), ("w1", w1), ("w2", w2), ("head", head), ("p", p))}
    t = v["x"]
    for j in range(topk):
        zz = (v["w1"][ids[:, j]] @ v["x"][:, :, None])[:, :, 0]
        hh = torch.nn.functional.silu(zz[:, :inter]) * zz[:, inter:]
        t = t + v["p"][:, j:j + 1] * (v["w2"][ids[:, j]] @ hh[:, :, None])[:, :, 0]
    want = torch.nn.functional.cross_entropy(t @ v["head"].T, target, reduction="none", ignore_index=-100)
    (want.sum() / count).backward()

    off_by = (loss.cpu().double() - want.detach()).square().mean().sqrt()
    assert off_by <= 0.012 * max(1.0, float(want.detach().square().mean().sqrt())), off_by
    assert not loss.cpu()[~live].any()
    for name, got in (("head", dhead), ("w2", dw2), ("w1", dw1), ("x", dx), ("p", dp)):
        ref = v[name].grad
        err = float((got.cpu().double() - ref).norm() / ref.norm())
        assert err <= 0.029, f"d{name}: relative error {err:.4f}"
