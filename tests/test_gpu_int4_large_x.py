"""4-bit products of large x.

While every |x| is below 2^112 no sum within a group of 128 columns leaves FP32's
range: at most 128 (24 + 31) 2^112 < 2^125.  With scales of 2^-20 and the largest x,
255 2^104, a result is at most 1024 * 8 * 2^-20 * 2^112 < 2^106.
"""
import numpy as np
import pytest
import torch

from oracle import int4

pytestmark = pytest.mark.gpu


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("m", [1, 4, 16, 70])
@pytest.mark.parametrize("signs", ["one", "mixed"])
def test_below_the_bound(dev, m, group, signs):
    """Every x of the largest size below 2^112: finite, and off 64 bits by the sums'
    rounding alone (every product is exact; GROUP * 2 + 2 K / GROUP + 16 additions,
    each off by 2^-23 of (24 + 16 + code) |x| s summed)."""
    n, k = 40, 1024
    g = torch.Generator().manual_seed(m + group)
    codes = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8).numpy()
    codes[0], codes[1] = 15, 0
    scales = torch.full((k // group, n), 2.0 ** -20)
    x = torch.full((m, k), 255 * 2.0 ** 104)
    assert (x.to(torch.bfloat16).float() == x).all() and x.max() < 2.0 ** 112
    if signs == "mixed":
        x *= torch.randint(0, 2, (m, k), generator=g) * 2.0 - 1
    y = _fg8().gemm_bf16_int4(x.to(torch.bfloat16).to(dev), torch.from_numpy(int4.pack(codes)).to(dev), scales.to(dev),
                              out_dtype=torch.float32).cpu().double().numpy()
    xd = x.double().numpy()
    want = xd @ int4.values(codes, scales.numpy()).T
    size = np.abs(xd) @ (40.0 + codes).T * 2.0 ** -20
    assert np.isfinite(y).all()
    assert (np.abs(y - want) <= (2 * group + 2 * k / group + 16) * 2.0 ** -23 * size).all()


def test_one_larger_element(dev):
    """A lone x of 2^115 among ordinary ones is no threshold: its row is finite, and
    an infinite one, or a NaN, spoils its own row only."""
    n, k = 24, 256
    g = torch.Generator().manual_seed(9)
    codes = torch.randint(1, 16, (n, k), generator=g, dtype=torch.uint8).numpy()
    codes[:, 5] = 15
    x = torch.randn(6, k, generator=g)
    x[0, 5], x[2, 5], x[4, 5] = 2.0 ** 115, float("inf"), float("nan")
    y = _fg8().gemm_bf16_int4(x.to(torch.bfloat16).to(dev), torch.from_numpy(int4.pack(codes)).to(dev),
                              torch.ones(k // 128, n, device=dev), out_dtype=torch.float32).cpu()
    assert (y[0] == 7 * 2.0 ** 115).all()          # (what the others add is far below half a step)
    assert y[2].isnan().all() and y[4].isnan().all()
    assert y[1].isfinite().all() and y[3].isfinite().all() and y[5].isfinite().all()
