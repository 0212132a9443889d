"""A float dw of gemm_bf16_epilogue_backward is as exact as its type: dz behind
an activation reaches it in two BF16 parts.

Bounds, with u = 2^-24: the slope's terms are below |z| + 2 and off by 4e-6 of
that; dz less its two parts is below 2^-16 of it (half an ulp is 2^-8 relative
at most, twice); each of the two sums of m products of BF16 values is off by at
most 2 (m + 1) u of the sum of its absolute products, their sum by u.  (With dz
in one part each term would be off by up to 2^-8.)
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _slope(act, z):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p + z * p * (1 - p)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return (z > 0).double() if act == "relu" else torch.ones_like(z)


# m, n, k and dw's tile: k split or not, ends inside tiles, odd n, the big tile
CASES = [(1, 1, 8, 128), (5, 37, 40, 128), (200, 2048, 512, 128), (2100, 72, 1000, 128), (1000, 203, 264, 128),
         (300, 4096, 2056, 256), (300, 4099, 2056, 256)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,n,k,tile", CASES)
def test_float_dw(dev, m, n, k, tile, act):
    import moe_grouped_gemm_fp8_amd as fg8
    print(f"float dw {m}x{n}x{k} {act}", flush=True)
    assert fg8.bf16_tile_choice("dw", m, n, k)["bm"] == tile
    g = torch.Generator(device=dev).manual_seed(m + n)
    x, w, dy, z = (torch.randn(*s, generator=g, device=dev).to(BF16) for s in ((m, k), (n, k), (m, n + 3), (m, n)))
    dy = dy[:, :n]
    term = dy.double().abs() * (z.double().abs() + 2) * (4e-6 if act in ("silu", "gelu") else 0.0)
    dz = dy.double() * _slope(act, z.double())
    off = term + (2.0 ** -16 * (dz.abs() + term) if act in ("silu", "gelu") else 0.0)
    X, t = x.double().abs(), (lambda v: v.T.contiguous())
    want, size = t(dz) @ x.double(), t(dz.abs() + off) @ X
    # (the remainder's products are below 2^-8 of the first part's)
    err = t(off) @ X + 2 * (m + 1) * U * (1 + 2.0 ** -8) ** 2 * size + U * want.abs() + 1e-38
    for needs in ((True, True, True), (False, True, False)):
        dx, dw, db = fg8.gemm_bf16_epilogue_backward(dy, x, w, z, activation=act, dw_dtype=F32, needs=needs)
        bad = ~((dw.double() - want).abs() <= err)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"
        if needs[0]:         # dx and dbias as with a BF16 dw
            again = fg8.gemm_bf16_epilogue_backward(dy, x, w, z, activation=act)
            assert torch.equal(dx, again[0]) and torch.equal(db, again[2])


def test_infinite_dz_stays(dev):
    """Beside an infinity nothing is left over."""
    import moe_grouped_gemm_fp8_amd as fg8
    z = torch.full((1, 8), 20.0, dtype=BF16, device=dev)                 # slope 1
    dy = torch.tensor([[float("inf"), float("-inf"), 1.0, -3.38e38, 0.0, 2.0, float("nan"), -1.0]], device=dev).to(BF16)
    x = torch.ones(1, 8, dtype=BF16, device=dev)
    for act in ("silu", "gelu"):
        _, dw, _ = fg8.gemm_bf16_epilogue_backward(dy, x, torch.ones(8, 8, dtype=BF16, device=dev), z, activation=act, dw_dtype=F32)
        got, want = dw[:, 0].cpu(), dy[0].float().cpu()
        assert torch.equal(got[~want.isnan()].isinf(), want[~want.isnan()].isinf()) and bool(got[6].isnan())
        assert torch.equal(got[[0, 1, 4]], want[[0, 1, 4]]) and bool(((got - want)[[2, 3, 5, 7]].abs() <= 1e-5 * want[[2, 3, 5, 7]].abs()).all())
