"""The 4-bit oracle against hand-worked values and torch's BF16 rounding."""
import numpy as np
import torch

from oracle import int4


def test_by_hand():
    # amax 7: scale 1; halves go to even codes; the other group is all zeros
    w = np.zeros((2, 64), np.float32)
    w[0, :8] = [7, -7, 0.5, 1.5, -0.5, -2.5, 3.4999998, 6.5]
    w[1, 32:36] = [-14, 14, 7, 1]
    codes, scales = int4.quantize(w, 32)
    assert codes[0, :8].tolist() == [15, 1, 8, 10, 8, 6, 11, 14]
    assert scales.tolist() == [[1, 1], [1, 2]]
    assert codes[1, 32:36].tolist() == [1, 15, 12, 8]      # 3.5 to even, 0.5 to even
    assert (codes[:, 40:] == 8).all() and (codes[1, :32] == 8).all()
    v = int4.values(codes, scales)
    assert v[0, :8].tolist() == [7, -7, 0, 2, 0, -2, 3, 6] and v[1, 32:36].tolist() == [-14, 14, 8, 0]
    assert int4.pack(codes)[0, :4].tolist() == [15 + 16 * 1, 8 + 16 * 10, 8 + 16 * 6, 11 + 16 * 14]


def test_bf16_rounding():
    g = torch.Generator().manual_seed(3)
    v = torch.cat([torch.randn(5000, generator=g), torch.tensor([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -2.0 ** -130])])
    assert np.array_equal(int4.bf16(v.numpy()), v.to(torch.bfloat16).float().numpy())


def test_error_is_half_a_step():
    w = np.random.default_rng(0).normal(size=(9, 256)).astype(np.float32)
    for group in (32, 64, 128):
        for bf in (False, True):
            codes, scales = int4.quantize(w, group, bf)
            assert codes.min() >= 1 and codes.max() <= 15
            off = np.abs(int4.values(codes, scales) - w)
            # (a BF16 scale may be 2^-8 below amax / 7, and the largest weight 7 times that further off)
            assert (off <= np.repeat(scales.T, group, 1) * (0.5 + 7 * 2.0 ** -8 * bf) * (1 + 1e-6)).all()


def test_subnormal_scales():
    """amax of 8, 10, 17 and 24 of the smallest steps: scales of 1, 1, 2 and 3 of
    them, quotients past 7 limited to it."""
    for step, bf in ((2.0 ** -149, False), (2.0 ** -133, True)):
        w = np.zeros((4, 32), np.float32)
        for r, top in enumerate((8, 10, 17, 24)):
            w[r, :4] = np.array([top, -top, 4, -1], np.float64) * step
        codes, scales = int4.quantize(w, 32, bf)
        assert (scales[0] / np.float32(step)).tolist() == [1, 1, 2, 3]
        assert codes[:, :4].tolist() == [[15, 1, 12, 7], [15, 1, 12, 7], [15, 1, 10, 8], [15, 1, 9, 8]]
        assert (codes[:, 4:] == 8).all()
