"""How the gated products, the 4-bit weights and the loss are called: refusals of the
Python layer, another stream, two streams at once, workspaces of the caller."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def test_refusals(dev):
    fg8 = _fg8()
    x, w, z = (torch.zeros(*s, dtype=BF16, device=dev) for s in ((4, 64), (32, 64), (4, 32)))
    h, off = z[:, :16].contiguous(), torch.zeros(3, dtype=torch.int32, device=dev)
    e = w.view(2, 16, 64)
    q, s = torch.zeros(32, 32, dtype=torch.uint8, device=dev), torch.ones(2, 32, device=dev)
    t, f = torch.zeros(4, dtype=torch.int64, device=dev), torch.zeros(4, device=dev)
    wrong = [
        lambda: fg8.gemm_bf16_gated(x, w[:31].contiguous()),                    # an odd number of rows
        lambda: fg8.gemm_bf16_gated(x, w[:, :56].contiguous()),                 # another k
        lambda: fg8.gemm_bf16_gated(x, e),
        lambda: fg8.gemm_bf16_gated(x, w[:, ::2]),                              # not contiguous
        lambda: fg8.gemm_bf16_gated(x, w, out=z),                               # [m, 2 n] for [m, n]
        lambda: fg8.grouped_gemm_bf16_gated(x, w, off),
        lambda: fg8.grouped_gemm_bf16_gated(x, e, off[:2].contiguous()),
        lambda: fg8.gemm_bf16_gated_backward(z, x, w, z),                       # dh as wide as z
        lambda: fg8.gemm_bf16_gated_backward(h, x, w, h),
        lambda: fg8.gemm_bf16_gated_backward(h[:1].expand(4, 16), x, w, z),     # a broadcast gradient
        lambda: fg8.grouped_gemm_bf16_gated_backward(h, x, e, z[:3].contiguous(), off),
        lambda: fg8.gemm_bf16_int4(x, q, s[:, :31].contiguous()),
        lambda: fg8.gemm_bf16_int4(x, q[:, :16].contiguous(), s),
        lambda: fg8.gemm_bf16_int4(x, q[:31].contiguous(), s[:, :31].contiguous(), gated=True),
        lambda: fg8.gemm_bf16_int4(x, q, s, residual=x, gated=True),
        lambda: fg8.gemm_bf16_int4(x, q, s, bias=torch.zeros(31, device=dev)),
        lambda: fg8.grouped_gemm_bf16_int4(x, q, s, off),
        lambda: fg8.int4_dequantize(q, s[None]),
        lambda: fg8.int4_quantize(w, group=0),
        lambda: fg8.linear_cross_entropy(x, w, t[:3].contiguous()),
        lambda: fg8.linear_cross_entropy(x, w, t.cpu()),
        lambda: fg8.linear_cross_entropy_backward(f[:3].contiguous(), x, w, t, f),
        lambda: fg8.linear_cross_entropy_backward(f, x, w, t, f[:3].contiguous()),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} went through")
    types = [
        lambda: fg8.gemm_bf16_gated(x.float(), w),
        lambda: fg8.gemm_bf16_gated(x, w, out_dtype=torch.float16),
        lambda: fg8.gemm_bf16_int4(x, q.int(), s),
        lambda: fg8.gemm_bf16_int4(x, q, s.half()),
        lambda: fg8.int4_quantize(w.half()),
        lambda: fg8.int4_quantize(w, scale_dtype=torch.float16),
        lambda: fg8.linear_cross_entropy(x, w, t.float()),
        lambda: fg8.linear_cross_entropy_backward(f.double(), x, w, t, f),
    ]
    for i, call in enumerate(types):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"call {i} went through")
    for call in (lambda: fg8.int4_quantize(w, group=48), lambda: fg8.gemm_bf16_int4(x, q, s.view(1, 64)[:, :32].contiguous().repeat(4, 1)),
                 lambda: fg8.gemm_bf16_gated(x[:, :60].contiguous(), w[:, :60].contiguous()),
                 lambda: fg8.linear_cross_entropy(x[:, :60].contiguous(), w[:, :60].contiguous(), t)):
        with pytest.raises(fg8.Fg8Error):
            call()


def _calls(fg8, dev, seed):
    g = torch.Generator().manual_seed(seed)

    def rand(*s, scale=1.0):
        return (torch.randn(*s, generator=g) * scale).to(BF16).to(dev)
    x, w, dh = rand(40, 4096), rand(264, 4096, scale=1 / 64), rand(40, 132)        # products in several k ranges
    q, s = fg8.int4_quantize(w, group=128)
    head, t = rand(3001, 4096, scale=1 / 64), torch.randint(0, 3001, (40,), generator=g).to(dev)

    def run():
        h, z = fg8.gemm_bf16_gated(x, w, save_z=True)
        out = [h, z, *fg8.gemm_bf16_gated_backward(dh, x, w, z, dw_dtype=F32), fg8.gemm_bf16_int4(x, q, s, activation="silu", gated=True)]
        loss, lse = fg8.linear_cross_entropy(x, head, t)
        return out + [loss, lse, *fg8.linear_cross_entropy_backward(loss, x, head, t, lse)]
    return run


def test_streams(dev):
    """The same bits on another stream, and on two streams at once."""
    fg8 = _fg8()
    runs = [_calls(fg8, dev, i) for i in range(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                got.append(r())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(c, d) for c, d in zip(a, b))


def test_own_workspace(dev):
    """A caller's workspace serves call after call of any of them, and is refused
    where it is too small."""
    fg8 = _fg8()
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 4096, generator=g).to(BF16).to(dev)
    w = (torch.randn(264, 4096, generator=g) / 64).to(BF16).to(dev)
    t = torch.randint(0, 264, (40,), generator=g).to(dev)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    h, z = fg8.gemm_bf16_gated(x, w, save_z=True)
    loss, lse = fg8.linear_cross_entropy(x, w, t)
    dx, dw = fg8.gemm_bf16_gated_backward(h, x, w, z)
    dxl, dwl = fg8.linear_cross_entropy_backward(loss, x, w, t, lse)
    for _ in range(2):
        assert torch.equal(fg8.gemm_bf16_gated(x, w, workspace=ws), h)
        assert all(torch.equal(a, b) for a, b in zip(fg8.linear_cross_entropy(x, w, t, workspace=ws), (loss, lse)))
        assert all(torch.equal(a, b) for a, b in zip(fg8.gemm_bf16_gated_backward(h, x, w, z, workspace=ws), (dx, dw)))
        assert all(torch.equal(a, b) for a, b in zip(fg8.linear_cross_entropy_backward(loss, x, w, t, lse, workspace=ws), (dxl, dwl)))
        assert not ws[:4096].any(), "the counters are left at zero"
    small = torch.zeros(4096, dtype=torch.uint8, device=dev)
    for call in (lambda: fg8.gemm_bf16_gated(x, w, workspace=small), lambda: fg8.linear_cross_entropy(x, w, t, workspace=small),
                 lambda: fg8.gemm_bf16_gated_backward(h, x, w, z, workspace=small),
                 lambda: fg8.linear_cross_entropy_backward(loss, x, w, t, lse, workspace=small)):
        with pytest.raises(fg8.Fg8Error):
            call()


def test_poisoned_workspaces(dev):
    """Nothing is read from a workspace before it is written there."""
    fg8 = _fg8()
    g = torch.Generator().manual_seed(6)
    x = torch.randn(700, 256, generator=g).to(BF16).to(dev)
    w = (torch.randn(1001 * 2, 256, generator=g) / 16).to(BF16).to(dev)
    t = torch.randint(0, 2002, (700,), generator=g).to(dev)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=dev)      # NaN in either type
    ws[:4096] = 0
    h, z = fg8.gemm_bf16_gated(x, w, save_z=True)
    loss, lse = fg8.linear_cross_entropy(x, w, t)
    plain = [loss, lse, *fg8.gemm_bf16_gated_backward(h, x, w, z, dw_dtype=F32), *fg8.linear_cross_entropy_backward(loss, x, w, t, lse)]
    got = list(fg8.linear_cross_entropy(x, w, t, workspace=ws))
    ws[4096:] = 255
    got += fg8.gemm_bf16_gated_backward(h, x, w, z, dw_dtype=F32, workspace=ws)
    ws[4096:] = 255
    got += fg8.linear_cross_entropy_backward(loss, x, w, t, lse, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, plain))


def test_infinite_and_nan_rows_stay_in_their_rows(dev):
    fg8 = _fg8()
    g = torch.Generator().manual_seed(7)
    x = torch.randn(6, 512, generator=g).to(BF16)
    w = (torch.randn(64, 512, generator=g) / 16).to(BF16).to(dev)
    bad = x.clone()
    bad[1, 7], bad[4, 500] = float("nan"), float("inf")
    fine = torch.tensor([0, 2, 3, 5])
    q, s = fg8.int4_quantize(w, group=64)
    for f in (lambda a: fg8.gemm_bf16_gated(a, w), lambda a: fg8.gemm_bf16_int4(a, q, s),
              lambda a: fg8.gemm_bf16_int4(a, q, s, gated=True, activation="silu"),
              lambda a: fg8.linear_cross_entropy(a, w, torch.arange(6, device=dev))[0][:, None]):
        a, b = f(x.to(dev)).cpu(), f(bad.to(dev)).cpu()
        assert torch.equal(a[fine], b[fine])
        assert not b[1].isfinite().any() and not b[4].isfinite().any()
