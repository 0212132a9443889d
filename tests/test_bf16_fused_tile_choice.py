"""The tile rule of the gated products and the loss through the C ABI (no GPU
call), on a device of 256 compute units."""
import ctypes

import pytest

from moe_grouped_gemm_fp8_amd import _lib

CUS = 256
GATED, GATED_RUNS, LOSS, LOGITS, DX = _lib.BF16_FUSED_PRODUCTS


def choice(product, m, n, k, groups=1):
    c = _lib.bf16_tile_choice(product, m, n, k, groups, CUS)
    return c["bm"], c["bn"], c["splits"], c["persistent"]


def test_gated():
    assert choice(GATED, 1, 1000, 2048) == (16, 32, 1, 0)          # sixteen gate and sixteen up rows
    assert choice(GATED, 64, 2048, 7168) == (64, 64, 4, 0)
    assert choice(GATED, 512, 6400, 1024) == (128, 128, 1, 0)      # 400 tiles of 128 x 128
    assert choice(GATED, 8192, 2048, 7168) == (256, 256, 1, 1)
    assert choice(GATED_RUNS, 3000, 2048, 7168, 32) == (128, 128, 1, 0)
    assert choice(GATED_RUNS, 50021, 2048, 7168, 32) == (256, 256, 1, 1)


def test_loss():
    for product in (LOSS, LOGITS):
        assert choice(product, 61, 32003, 2048) == (64, 128, 1, 0)
        assert choice(product, 256, 32000, 4096) == (128, 128, 1, 0)
        assert choice(product, 8192, 128000, 7168) == (256, 256, 1, 1)
    assert choice(DX, 4095, 100003, 2048) == (256, 256, 2, 1)      # two ranges of a piece's classes


def test_the_workspace_holds_the_splits():
    for m, n, k in ((64, 2048, 7168), (20, 72, 2056), (300, 264, 328)):
        bm, bn, splits, _ = choice(GATED, m, n, k)
        tiles = -(-m // bm) * -(-2 * n // bn)
        assert _lib.lib().fg8_gemm_bf16_gated_workspace_bytes(m, n, k) == (4096 + tiles * splits * bm * bn * 4 if splits > 1 else 0)
    for m, v, k in ((40, 1000, 64), (53, 300, 2048), (700, 16600, 72)):
        bm, bn, splits, _ = choice(LOSS, m, v, k)
        tiles = -(-v // bn)
        product = -(-m // bm) * tiles * splits * bm * bn * 4 if splits > 1 else 0
        assert _lib.lib().fg8_linear_cross_entropy_workspace_bytes(m, v, k) == 4096 + product + -(-m * 4 // 16) * 16 + tiles * m * 8


@pytest.mark.parametrize("args", [(5, 8, 8, 8, 1, 256), (-1, 8, 8, 8, 1, 256), (0, 0, 8, 8, 1, 256), (0, 8, 0, 8, 1, 256), (2, 8, 8, 0, 1, 256),
                                  (0, 8, 8, 8, 2, 256), (1, 8, 8, 8, 0, 256), (1, 8, 8, 8, 1025, 256), (4, 8, 8, 8, 2, 256),
                                  (0, 8, 8, 8, 1, 0), (3, 1 << 31, 8, 8, 1, 256), (2, 8, (1 << 22) + 1, 8, 1, 256),
                                  (0, 8, (1 << 21) + 1, 8, 1, 256)])
def test_refusals(args):
    out = (ctypes.c_int32 * 4)()
    assert _lib.lib().fg8_bf16_fused_tile_choice(*args, ctypes.cast(out, ctypes.c_void_p)) == 1
    assert _lib.lib().fg8_bf16_fused_tile_choice(0, 8, 8, 8, 1, 256, None) == 1


def test_the_largest_sizes():
    for product in _lib.BF16_FUSED_PRODUCTS:
        _lib.bf16_tile_choice(product, (1 << 31) - 1024, 1 << 21, 1 << 22, 1, CUS)
