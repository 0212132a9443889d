"""Sizes past what one launch can hold (fewer than 2^32 threads) are refused by
the C ABI as unsupported before anything is launched."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED = 0, 1, 2
MOST = (2 ** 32 - 1) // 256          # workgroups of 256 threads


@pytest.fixture(scope="module")
def L():
    from moe_grouped_gemm_fp8_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfg8.so is not built (run __graft_entry__.build())")
    return _lib.lib()


ok = P(0x10000)      # never dereferenced: nothing here is launched


@pytest.mark.parametrize("bf16,span", [(1, 512), (0, 256)])
def test_combine(L, bf16, span):
    """A wave takes a span of a token's columns, four waves a workgroup."""
    for spans in (1, 3):
        tokens = 4 * MOST // spans + 1
        hidden = span * (spans - 1) + 8
        assert L.moe_combine(ok, bf16, 8, ok, ok, None, tokens, 2, hidden, ok, None) == EUNSUPPORTED
        assert b"exceed a launch" in L.fg8_last_error()
        # the largest that a launch holds gets past this check, to the next one
        assert L.moe_combine(None, bf16, 8, ok, ok, None, 4 * MOST // spans, 2, hidden, ok, None) == EINVAL
    for tokens in (1 << 31, 1 << 40, 1 << 62):
        assert L.moe_combine(ok, bf16, 8, ok, ok, None, tokens, 2, 64, ok, None) == EUNSUPPORTED


def test_combine_backward(L):
    """A workgroup a token, and one for four rows."""
    def call(tokens, rows, y=ok):
        return L.moe_combine_backward(ok, y, 1, rows, ok, ok, ok, tokens, 2, 8, ok, ok, None)
    for tokens, rows in ((MOST, 1), (MOST - 1, 5), (1, 4 * MOST - 3), (0, 4 * MOST + 1), (1 << 31, 1), (1 << 62, 1)):
        assert call(tokens, rows) == EUNSUPPORTED, (tokens, rows)
    for tokens, rows in ((MOST - 1, 4), (1, 4 * MOST - 4), (0, 4 * MOST)):
        assert call(tokens, rows, y=None) == EINVAL, (tokens, rows)


def test_products(L):
    """A workgroup of 256 threads for every tile: 131072 rows over 1024 experts
    are 2049 row tiles of 128 at most."""
    n = 1 << 22
    assert L.grouped_gemm_bf16(ok, 64, ok, ok, ok, n, 1, 131072, n, 64, 1024, None) == EUNSUPPORTED
    assert b"exceed a launch" in L.fg8_last_error()
    assert L.grouped_gemm_bf16_dgrad(ok, 64, ok, ok, ok, n, 1, 131072, 64, n, 1024, None) == EUNSUPPORTED
    # 32768 x 1024 tiles of a weight gradient, for each of four experts (short
    # runs: long ones take a launch of one workgroup a CU, which has no such limit)
    assert L.grouped_gemm_bf16_wgrad(ok, n, ok, 1 << 18, ok, ok, 0, 2, n, 1 << 18, 4, None) == EUNSUPPORTED
    assert b"exceed a launch" in L.fg8_last_error()


def test_row_strides(L):
    """No ld past 2^22, an output's or a normed row's either."""
    far, n = (1 << 22) + 8, 1 << 22
    assert L.grouped_gemm_bf16(ok, 64, ok, ok, ok, far, 1, 10, 64, 64, 4, None) == EUNSUPPORTED
    assert L.grouped_gemm_bf16_dgrad(ok, 64, ok, ok, ok, far, 1, 10, 64, 64, 4, None) == EUNSUPPORTED
    assert L.gemm_bf16_epilogue(ok, 64, ok, None, 0, 0, ok, far, None, ok, 64, 1, 1024, 64, 64, None, 0, None) == EUNSUPPORTED
    assert L.gemm_bf16_epilogue(ok, 64, ok, None, 0, 0, None, 0, None, ok, n + 8, 1, 1024, n + 8, 64, None, 0, None) == EUNSUPPORTED
    assert L.gemm_bf16_epilogue_backward(ok, far, ok, 64, ok, ok, 3, ok, ok, 1, ok, 8, 64, 64, ok, 1 << 30, None) == EUNSUPPORTED
    assert L.layer_norm(ok, far, 1, ok, None, 0, 1e-5, 4, 64, ok, ok, ok, None) == EUNSUPPORTED
    assert L.layer_norm_backward(ok, far, ok, 64, 1, ok, 0, ok, ok, 4, 64, ok, ok, ok, ok, 1 << 20, None) == EUNSUPPORTED
