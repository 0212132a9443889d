"""The BF16 products' tile rule through the C ABI (no GPU call), on a device of
256 compute units."""
import ctypes

import pytest

from moe_grouped_gemm_fp8_amd import _lib

CUS = 256
FORWARD, DX, DW, GROUPED, DGRAD, WGRAD = _lib.BF16_PRODUCTS


def choice(product, m, n, k, groups=1):
    c = _lib.bf16_tile_choice(product, m, n, k, groups, CUS)
    return c["bm"], c["bn"], c["splits"], c["persistent"]


def test_few_rows():
    assert choice(FORWARD, 1, 1024, 2048) == (16, 16, 1, 0)          # both operands straight into registers
    assert choice(FORWARD, 64, 2112, 7168) == (64, 64, 7, 0)         # 33 tiles, k split over the device
    assert choice(GROUPED, 40, 1024, 2048, 8) == (16, 16, 1, 0)


def test_many_rows():
    assert choice(FORWARD, 8191, 7168, 2048) == (256, 256, 1, 1)
    assert choice(DW, 4096, 7168, 2048) == (256, 256, 1, 1)
    assert choice(GROUPED, 50021, 4096, 7168, 32) == (256, 256, 1, 1)


def test_the_workspace_is_the_splits():
    """One FP32 tile a split, behind the counters."""
    for m, n, k in ((64, 2112, 7168), (33, 70, 1000), (200, 264, 2048), (4096, 4096, 512)):
        bm, bn, splits, _ = choice(FORWARD, m, n, k)
        tiles = -(-m // bm) * -(-n // bn)
        assert _lib.lib().fg8_gemm_bf16_workspace_bytes(m, n, k) == (4096 + tiles * splits * bm * bn * 4 if splits > 1 else 0)


@pytest.mark.parametrize("args", [(6, 8, 8, 8, 1, 256), (-1, 8, 8, 8, 1, 256), (0, 0, 8, 8, 1, 256), (0, 8, 0, 8, 1, 256),
                                  (0, 8, 8, 0, 1, 256), (0, 8, 8, 8, 2, 256), (3, 8, 8, 8, 0, 256), (3, 8, 8, 8, 1025, 256),
                                  (0, 8, 8, 8, 1, 0), (0, 1 << 31, 8, 8, 1, 256)])
def test_refusals(args):
    out = (ctypes.c_int32 * 4)()
    assert _lib.lib().fg8_bf16_tile_choice(*args, ctypes.cast(out, ctypes.c_void_p)) == 1
    assert _lib.lib().fg8_bf16_tile_choice(0, 8, 8, 8, 1, 256, None) == 1
