"""The erf GELU and its slope to FP32 accuracy, relative accuracy in the lower
tail included.

z reaches the activation exactly: a product of one-term or two-term sums of BF16
values that do not overlap, and, backward, the saved z itself with a single row,
whose column sum is dz before its rounding.

Bounds, with u = 2^-24.  For z < 0 the kernels compute Phi(z) as
e^(-z^2 / 2) t p(t): t is off by 3 u relative (a rounding and a reciprocal of one
ulp), which t p(t) passes on at most 2.61-fold; p's eight terms are evaluated with
8 roundings of at most 1.74 of its value each, their constants with one more; the
fit adds 1.2e-7, exp2 and the two products 4 u; the exponent z^2 / 2 is off by
three roundings, 1.5 u z^2.  Together r(z) = 1.9e-6 + 9e-8 z^2, relative.  For
z >= 0, 1 - Phi(-z) adds u.  The last products round to FP32: 2 u relative.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _phi(z):
    return np.array([math.erfc(-v / math.sqrt(2)) / 2 for v in z])


def _relative(z):
    return 1.9e-6 + 9e-8 * z * z


def _grid():
    """Values of 16 significand bits, as two BF16 parts."""
    g = torch.Generator().manual_seed(31)
    z = torch.cat([torch.linspace(-12, 6, 8191), torch.randn(8000, generator=g), torch.tensor([0.0, -0.0, 1e-30, -1e-30])])
    hi = z.to(BF16)
    lo = (z - hi.float()).to(BF16)
    return hi, lo, hi.double().add(lo.double()).numpy()


def test_gelu(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    hi, lo, z = _grid()
    x = torch.zeros(len(z), 8, dtype=BF16)
    x[:, 0], x[:, 1] = hi, lo
    w = torch.zeros(1, 8, dtype=BF16)
    w[0, :2] = 1
    y = fg8.gemm_bf16_epilogue(x.to(dev), w.to(dev), activation="gelu", out_dtype=F32)[:, 0].cpu().double().numpy()
    tail = _phi(-np.abs(z))
    want = z * _phi(z)
    err = np.abs(z) * (tail * _relative(z) + np.where(z < 0, 0, U)) + 2 * U * np.abs(want) + 1e-38
    off = np.abs(y - want) / err
    assert off.max() <= 1, f"z = {z[off.argmax()]}: {y[off.argmax()]} for {want[off.argmax()]}, {off.max():.2f} times the bound"


def test_gelu_slope(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    hi, _, _ = _grid()
    n = len(hi) // 8 * 8
    z = hi[:n].double().numpy()
    one = torch.ones(1, n, dtype=BF16, device=dev)
    _, _, db = fg8.gemm_bf16_epilogue_backward(one, torch.zeros(1, 8, dtype=BF16, device=dev),
                                               torch.zeros(n, 8, dtype=BF16, device=dev), z=hi[:n].reshape(1, n).to(dev),
                                               activation="gelu", needs=(False, False, True))
    tail, bell = _phi(-np.abs(z)), np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    want = _phi(z) + z * bell
    # the density's exponent as above, its constant and products 6 u; the last sum rounds once
    err = (tail * _relative(z) + np.where(z < 0, 0, U) + np.abs(z) * bell * (6 * U + 9e-8 * z * z) + U * np.abs(want) + 1e-38)
    off = np.abs(db.cpu().double().numpy() - want) / err
    assert off.max() <= 1, f"z = {z[off.argmax()]}: {off.max():.2f} times the bound"
