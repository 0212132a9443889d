"""The gated products, the 4-bit weights and the loss on tensors past 2^31 elements:
what lies behind them, against float32 products of the same values on the GPU.

Sums of K products in FP32, both sides: 4 (K + 1) 2^-24 of the absolute sums between
them, and 2^-8 of the value for a BF16 output.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def empty_cache():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _normal(g, *shape, scale=1.0):
    return torch.empty(*shape, dtype=BF16, device="cuda").normal_(0, scale, generator=g)


def _close(got, want, size, k):
    bound = 4 * (k + 1) * 2.0 ** -24 * size + (2.0 ** -8 * want.abs() if got.dtype == BF16 else 0) + 1e-30
    assert ((got.float() - want).abs() <= bound).all(), float(((got.float() - want).abs() / bound).max())


def test_gated_z_past_2_31(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    print("gated, z of 530,000 x 4112", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    m, n, k = 530000, 2056, 64
    x, w = _normal(g, m, k), _normal(g, 2, 2 * n, k, scale=0.125)
    off = torch.tensor([0, 400000, m - 3], dtype=torch.int32, device=dev)
    h, z = fg8.grouped_gemm_bf16_gated(x, w, off, activation="none", save_z=True)
    assert z.numel() > 1 << 31
    for r, e in ((slice(399990, 400000), 0), (slice(400000, 400010), 1), (slice(m - 13, m - 3), 1)):
        want = x[r].float() @ w[e].float().T
        size = x[r].float().abs() @ w[e].float().abs().T
        _close(z[r], want, size, k)
        hw = want[:, :n] * want[:, n:]
        off_by = (h[r].float() - hw).abs()
        es = 4 * (k + 1) * 2.0 ** -24 * size
        assert (off_by <= es[:, :n] * want[:, n:].abs() + (want[:, :n].abs() + es[:, :n]) * es[:, n:] + 2.0 ** -8 * hw.abs() + 1e-30).all()
    assert not z[m - 3:].any() and not h[m - 3:].any()
    dh = _normal(g, 10, n)
    dx, _ = fg8.grouped_gemm_bf16_gated_backward(h, x, w, z, off, activation="none", needs=(True, False))
    r = slice(m - 13, m - 3)
    dz = torch.cat([h[r].float() * z[r, n:].float(), h[r].float() * z[r, :n].float()], 1)
    want, size = dz @ w[1].float(), dz.abs() @ w[1].float().abs()
    assert ((dx[r].float() - want).abs() <= (2.0 ** -8 + 4 * (2 * n + 1) * 2.0 ** -24) * size + 2.0 ** -8 * want.abs()).all()
    assert not dx[m - 3:].any()
    del dh


def test_int4_codes_past_2_31(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    print("int4, 40 experts of 16384 x 8192", flush=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    e, n, k = 40, 16384, 8192
    q = torch.empty(e, n, k // 2, dtype=torch.uint8, device=dev)
    q.random_(0, 256, generator=g)
    scales = torch.rand(e, k // 32, n, device=dev, generator=g)
    assert q.numel() > 1 << 31
    x = _normal(g, 5, k)
    off = torch.zeros(e + 1, dtype=torch.int32, device=dev)
    off[-2:] = torch.tensor([2, 5], dtype=torch.int32)            # rows 0 and 1 of expert 38, the others of 39
    y = fg8.grouped_gemm_bf16_int4(x, q, scales, off, out_dtype=F32)
    back = torch.empty(2, n, k, dtype=F32, device=dev)
    back.copy_(fg8.int4_dequantize(q[-2:], scales[-2:], out_dtype=F32))
    for j, r in ((0, slice(0, 2)), (1, slice(2, 5))):
        # (16 + code and 24 for a code's 8 at most: five times the sums)
        _close(y[r], x[r].float() @ back[j].T, 5 * (x[r].float().abs() @ (back[j].abs() + 8 * scales[j - 2].T.repeat_interleave(32, 1)).T), k)
    w = _normal(g, 33, n, 4096)
    assert w.numel() > 1 << 31
    q, scales = fg8.int4_quantize(w, group=128, scale_dtype=BF16)
    last, s = fg8.int4_quantize(w[-1:].contiguous(), group=128, scale_dtype=BF16)
    assert torch.equal(q[-1], last[0]) and torch.equal(scales[-1], s[0])


def test_head_past_2_31(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    print("loss, 3,000,000 classes of 768", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    m, v, k = 40, 3000000, 768
    x, w = _normal(g, m, k), _normal(g, v, k, scale=0.1)
    assert w.numel() > 1 << 31
    t = torch.randint(v - 100, v, (m,), device=dev, generator=g)
    loss, lse = fg8.linear_cross_entropy(x, w, t)
    logits = x.float() @ w.float().T
    want = torch.logsumexp(logits.double(), 1)
    at = torch.arange(m, device=dev)
    e = 4 * (k + 1) * 2.0 ** -24 * float((x.float().abs().sum(1) * 0.6).max())
    # (the classes' sum in any order: V 2^-24 at most, far less by its size)
    assert ((lse - want).abs() <= e + 2.0 ** -17 + 2.0 ** -22 * want.abs()).all()
    assert ((loss - (want - logits[at, t])).abs() <= 2 * e + 2.0 ** -16 + 2.0 ** -21 * want.abs()).all()
    dx, dw = fg8.linear_cross_entropy_backward(torch.ones(m, device=dev), x, w, t, lse, dw_dtype=BF16)
    dl = torch.exp(logits[:, -200:] - lse[:, None])
    dl[at, t - (v - 200)] -= 1
    want, size = dl.T @ x.float(), dl.abs().T @ x.float().abs()
    assert ((dw[-200:].float() - want).abs() <= (2.0 ** -8 + e + 2.0 ** -16) * size + 2.0 ** -8 * want.abs() + 1e-12).all()


def test_most_classes(dev):
    """As many classes as a head may have, few rows: pieces of the vocabulary whose
    dx is added up by the tiles of few rows."""
    import moe_grouped_gemm_fp8_amd as fg8
    print("loss backward, 100 rows, 2^22 classes of 16", flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    m, v, k = 100, 1 << 22, 16
    assert 2 * m * v > 512 << 20
    x, w = _normal(g, m, k), _normal(g, v, k)
    t = torch.randint(0, v, (m,), device=dev, generator=g)
    loss, lse = fg8.linear_cross_entropy(x, w, t)
    logits = x.float() @ w.float().T
    want = torch.logsumexp(logits.double(), 1)
    e = 4 * (k + 1) * 2.0 ** -24 * float((x.float().abs() @ w.float().abs().amax(0)).max())
    assert ((lse - want).abs() <= e + 2.0 ** -17 + 2.0 ** -22 * want.abs()).all()
    dx, dw = fg8.linear_cross_entropy_backward(torch.ones(m, device=dev), x, w, t, lse, dw_dtype=BF16)
    dl = torch.exp(logits - lse[:, None])
    dl[torch.arange(m, device=dev), t] -= 1
    size = dl.abs() @ w.float().abs()
    # (float32 sums of 2^22 terms on both sides, in blocks: 2^-24 of the absolute sums
    # for each of some thousand additions in a row at most)
    assert ((dx.float() - dl @ w.float()).abs() <= (2.0 ** -8 + e + 2.0 ** -12) * size + 2.0 ** -8 * (dl @ w.float()).abs()).all()
    some = torch.cat([t[:20], torch.tensor([0, 2097151, 2097152, v - 1], device=dev)])
    want, size = dl[:, some].T @ x.float(), dl[:, some].abs().T @ x.float().abs()
    assert ((dw[some].float() - want).abs() <= (2.0 ** -8 + e + 2.0 ** -16) * size + 2.0 ** -8 * want.abs() + 1e-12).all()
