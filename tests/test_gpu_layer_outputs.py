"""Layer norm's y where the mean is far from zero.

With u = 2^-24 and C columns the kernel's mean is off by at most (C + 2) u
mean|x|, its rstd by at most 0.04 at this input (the mean's error squared over
the variance, halved, below 0.035, and rounding); y passes on (x - mean) times
rstd's error and rstd times the mean's.  Against the kernel's own mean and rstd
y is three rounded operations: 3 u of its value.
"""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("cols", [1024, 7169])
def test_y_of_a_far_mean(dev, cols):
    import moe_grouped_gemm_fp8_amd as fg8
    far = 4096.0 * 1024 / cols                  # the same (C + 2) u far for both
    x = far + torch.randn(8, cols, generator=torch.Generator().manual_seed(2))
    X = x.double().numpy()
    y0, m0, r0 = layer.layer_norm(X, np.ones(cols), None, 0.0)
    y, mean, rstd = (t.cpu().double().numpy() for t in fg8.layer_norm(x.to(dev), torch.ones(cols, device=dev), None, 0.0))
    own = (X - mean[:, None]) * rstd[:, None]
    assert (np.abs(y - own) <= 3 * U * np.abs(own)).all()
    e_m = (cols + 2) * U * np.abs(X).mean(1, keepdims=True) + U * np.abs(X)
    e_r = 0.04
    err = np.abs(y0) / r0[:, None] * e_r + e_m * (r0[:, None] + e_r) + 3 * U * np.abs(y0)
    assert (np.abs(y - y0) <= err).all()
