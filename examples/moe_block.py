"""One MoE block in BF16, forward and backward, on the library's entry points:

    h   = layer_norm(x)
    p   = softmax over the top-k of h Wr^T + br           (router)
    s   = gelu(h Ws1^T + bs1) Ws2^T + bs2 + x             (shared expert, on the residual stream)
    out = s + sum_j p_j relu(h W1_e^T) W2_e^T             (routed experts e of the token)

The router's logits, the shared expert and its biases go through
gemm_bf16_epilogue, the routing layout through moe_contiguous_layout_fp8 (its
row maps; the FP8 rows are there for a forward pass in FP8), the routed experts
through grouped_gemm_bf16 and its two gradients, and the way back to the tokens
through moe_combine.  The backward pass is written out by hand.

    python examples/moe_block.py [tokens]      times one forward and backward pass
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_fp8_amd as fg8  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class MoeBlock:
    def __init__(self, hidden, inter, experts, topk, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.experts, self.topk = experts, topk

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).to(BF16).to(device)

        def vector(n, around=0.0):
            return (around + 0.1 * torch.randn(n, generator=g)).to(device)

        self.norm_w, self.norm_b = vector(hidden, 1.0), vector(hidden)
        self.wr, self.br = weight(experts, hidden), vector(experts)
        self.ws1, self.bs1 = weight(inter, hidden), vector(inter)
        self.ws2, self.bs2 = weight(hidden, inter), vector(hidden)
        self.w1, self.w2 = weight(experts, inter, hidden), weight(experts, hidden, inter)

    def forward(self, x):
        """x bf16 [tokens, hidden] -> (out bf16 [tokens, hidden], what backward needs)."""
        h, mean, rstd = fg8.layer_norm(x, self.norm_w, self.norm_b)
        logits = fg8.gemm_bf16_epilogue(h, self.wr, self.br, out_dtype=F32)
        top, ids = logits.topk(self.topk, dim=1)
        p = torch.softmax(top, 1)
        lay = fg8.moe_contiguous_layout_fp8(h, ids.to(torch.int32), self.experts)
        # the layout's rows in BF16: each row's token, zeros in padding rows
        token = lay["row_token"].long()
        rows = torch.where((token >= 0)[:, None], h[token.clamp(min=0)], 0)
        off = lay["expert_offsets"]
        z1 = fg8.grouped_gemm_bf16(rows, self.w1, off)
        a1 = z1.clamp(min=0)
        y = fg8.grouped_gemm_bf16(a1, self.w2, off)
        a, za = fg8.gemm_bf16_epilogue(h, self.ws1, self.bs1, activation="gelu", save_z=True)
        s = fg8.gemm_bf16_epilogue(a, self.ws2, self.bs2, residual=x)
        out = fg8.moe_combine(y, lay["token_row"], p, residual=s)
        return out, (x, h, mean, rstd, ids, p, lay, token, rows, z1, a1, y, a, za)

    def backward(self, dout, saved):
        """dout bf16 [tokens, hidden] -> (dx, gradients by parameter name)."""
        x, h, mean, rstd, ids, p, lay, token, rows, z1, a1, y, a, za = saved
        off, grads = lay["expert_offsets"], {}
        dy, dp = fg8.moe_combine_backward(dout, y, lay["token_row"], lay["row_token"], p)
        # routed experts
        grads["w2"] = fg8.grouped_gemm_bf16_wgrad(dy, a1, off)
        dz1 = fg8.grouped_gemm_bf16_dgrad(dy, self.w2, off) * (z1 > 0)
        grads["w1"] = fg8.grouped_gemm_bf16_wgrad(dz1, rows, off)
        drows = fg8.grouped_gemm_bf16_dgrad(dz1, self.w1, off, out_dtype=F32)
        # each token's rows back onto it, with weight 1
        dh = fg8.moe_combine(drows, lay["token_row"], torch.ones_like(p))
        # shared expert
        da, grads["ws2"], grads["bs2"] = fg8.gemm_bf16_epilogue_backward(dout, a, self.ws2, dw_dtype=F32)
        dhs, grads["ws1"], grads["bs1"] = fg8.gemm_bf16_epilogue_backward(da, h, self.ws1, za, activation="gelu", dw_dtype=F32)
        # router: softmax over the chosen logits
        dtop = p * (dp - (p * dp).sum(1, keepdim=True))
        dlogits = torch.zeros(x.shape[0], self.experts, device=x.device).scatter_(1, ids, dtop).to(BF16)
        dhr, grads["wr"], grads["br"] = fg8.gemm_bf16_epilogue_backward(dlogits, h, self.wr, dw_dtype=F32)
        dh = (dh + dhs + dhr).to(BF16)
        dx, grads["norm_w"], grads["norm_b"] = fg8.layer_norm_backward(dh, x, self.norm_w, mean, rstd)
        return dx + dout, grads


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 8192
    block = MoeBlock(hidden=2048, inter=1536, experts=32, topk=8)
    x = torch.randn(tokens, 2048, device="cuda").to(BF16)
    dout = torch.randn(tokens, 2048, device="cuda").to(BF16)
    for _ in range(3):
        block.backward(dout, block.forward(x)[1])
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(10):
        block.backward(dout, block.forward(x)[1])
    torch.cuda.synchronize()
    each = (time.perf_counter() - start) / 10
    # the routed experts' two products, forward and twice backward
    flops = 6 * tokens * block.topk * 2 * 2048 * 1536
    print(f"{tokens} tokens: {each * 1e3:.2f} ms a forward and backward pass, "
          f"{flops / each / 1e12:.0f} TFLOP/s of routed products")


if __name__ == "__main__":
    main()
