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


BIG, DUO, MID = (256, 256, 1, 1), (128, 256, 1, 0), (128, 128, 1, 0)


@pytest.mark.parametrize("m,n,k", [(2048, 4096, 7168), (4096, 2048, 7168), (1024, 7168, 2048)])
def test_dense_small_tiles_while_one_round_holds_them(m, n, k):
    """Up to two 128 x 128 tiles a CU, for y and for gradients of that size:
    the big tile measured 6 to 17% slower there."""
    assert choice(FORWARD, m, n, k) == MID
    assert choice(DX, m, k, n) == MID               # dx [m][n], summed over k
    assert choice(DW, k, m, n) == MID               # dw [m][n], summed over k


@pytest.mark.parametrize("m,n,k", [(1280, 7168, 2048), (4096, 2560, 7168), (4000, 5000, 2048), (8192, 8192, 8192)])
def test_dense_big_tiles_from_a_second_round_on(m, n, k):
    assert choice(FORWARD, m, n, k) == BIG
    assert choice(DX, m, k, n) == BIG
    assert choice(DW, k, m, n) == BIG


def test_the_backward_pass_of_4096x7168x2048():
    assert choice(DX, 4096, 7168, 2048) == MID and choice(DW, 4096, 7168, 2048) == BIG


@pytest.mark.parametrize("runs,rows,n,k,tile", [
    (8, 4096, 4096, 2048, BIG), (2, 8192, 4096, 4096, BIG), (8, 1024, 4096, 2048, BIG), (16, 1024, 7168, 2048, BIG),
    (32, 512, 7168, 2048, BIG),                                              # long runs, two tiles a CU and more
    (16, 250, 4096, 2048, DUO), (32, 64, 7168, 2048, DUO),                   # short runs of many tiles
    (8, 512, 4096, 2048, MID), (4, 1024, 4096, 2048, MID), (16, 1024, 2048, 1024, MID), (2, 4096, 2048, 2048, MID)])
def test_weight_gradients_of_runs(runs, rows, n, k, tile):
    assert choice(WGRAD, runs * rows, n, k, runs) == tile


def test_row_runs_from_half_the_device_on():
    for product, n, k in ((GROUPED, 2048, 1024), (DGRAD, 1024, 2048)):
        assert choice(product, 8 * 512, n, k, 8) == BIG                     # 128 by the average
        assert choice(product, 8 * 256, n, k, 8) != BIG                     # 64
