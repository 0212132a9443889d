"""The C ABI of the BF16 products, layer norm and the combine step without a
GPU: refusals that come before any launch, and the calls on nothing."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from moe_grouped_gemm_fp8_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfg8.so is not built (run __graft_entry__.build())")
    return _lib.lib()


ok, odd = P(0x10000), P(0x10008)      # never dereferenced: nothing here is launched


def test_grouped(L):
    for f in (L.grouped_gemm_bf16, L.grouped_gemm_bf16_dgrad):
        def call(x=ok, ldx=64, w=ok, off=ok, y=ok, ldy=64, out=1, rows=10, n=64, k=64, e=4):
            return f(x, ldx, w, off, y, ldy, out, rows, n, k, e, None)
        for a in ({"x": None}, {"w": None}, {"off": None}, {"y": None}, {"x": odd}, {"y": odd}, {"out": 2}, {"rows": -1},
                  {"rows": 1 << 31}, {"n": 0}, {"k": 0}, {"e": 0}, {"e": 1025}, {"ldx": 56}, {"ldx": 68}, {"ldy": 63}):
            assert call(**a) == EINVAL, a
        assert call(k=60) == EUNSUPPORTED and call(ldx=(1 << 22) + 8) == EUNSUPPORTED
        assert call(k=1 << 23, ldx=1 << 23, ldy=1 << 23) == EUNSUPPORTED
        assert call(rows=0, x=None, w=None, y=None) == OK
    assert L.grouped_gemm_bf16_dgrad(ok, 64, ok, ok, ok, 64, 1, 10, 60, 64, 4, None) == EUNSUPPORTED
    f = L.grouped_gemm_bf16_wgrad
    assert f(None, 64, ok, 64, ok, ok, 0, 10, 64, 64, 4, None) == EINVAL
    assert f(ok, 64, ok, 64, None, ok, 0, 10, 64, 64, 4, None) == EINVAL
    assert f(ok, 64, ok, 64, ok, ok, 0, 10, 63, 64, 4, None) == EUNSUPPORTED
    assert f(ok, 63, ok, 64, ok, ok, 0, 10, 64, 64, 4, None) == EINVAL
    assert b"lddy" in L.fg8_last_error()


def test_dense(L):
    def call(x=ok, ldx=7168, w=ok, bias=None, bb=0, act=0, res=None, ldr=520, z=None, y=ok, ldy=520, out=1, m=40, n=520,
             k=7168, ws=None, size=0):
        return L.gemm_bf16_epilogue(x, ldx, w, bias, bb, act, res, ldr, z, y, ldy, out, m, n, k, ws, size, None)
    need = L.fg8_gemm_bf16_workspace_bytes(40, 520, 7168)
    assert need > 4096
    for a in ({"x": None}, {"w": odd}, {"y": None}, {"bias": odd}, {"z": odd}, {"bb": 2}, {"act": 4}, {"act": -1}, {"m": -1},
              {"res": ok, "ldr": 519}, {"res": odd}, {"ldy": 519}, {"out": 3}, {}, {"ws": ok, "size": need - 1},
              {"ws": odd, "size": need}):
        assert call(**a) == EINVAL, a
    assert b"workspace" in L.fg8_last_error()
    assert call(k=7164) == EUNSUPPORTED
    assert call(m=0, x=None, w=None, y=None) == OK

    def back(dy=ok, lddy=64, x=ok, ldx=64, w=ok, z=ok, act=3, dx=ok, dw=ok, out=1, db=ok, m=8, n=64, k=64, ws=ok, size=1 << 30):
        return L.gemm_bf16_epilogue_backward(dy, lddy, x, ldx, w, z, act, dx, dw, out, db, m, n, k, ws, size, None)
    for a in ({"dy": None}, {"z": None}, {"w": None}, {"x": None}, {"dx": None, "dw": None, "db": None}, {"act": 9}, {"m": 0},
              {"ws": None}, {"size": L.fg8_gemm_bf16_backward_workspace_bytes(8, 64, 64) - 1}, {"lddy": 63}, {"ldx": 60}):
        assert back(**a) == EINVAL, a
    assert back(k=60) == EUNSUPPORTED


def test_row_limit(L):
    # rows rounded up to a tile have to fit 32 bits
    most = (1 << 31) - 1024
    for rows, status in ((most + 1, EUNSUPPORTED), ((1 << 31) - 1, EUNSUPPORTED)):
        assert L.grouped_gemm_bf16(ok, 64, ok, ok, ok, 64, 1, rows, 64, 64, 4, None) == status
        assert L.grouped_gemm_bf16_dgrad(ok, 64, ok, ok, ok, 64, 1, rows, 64, 64, 4, None) == status
        assert L.grouped_gemm_bf16_wgrad(ok, 64, ok, 64, ok, ok, 1, rows, 64, 64, 4, None) == status
        assert L.gemm_bf16_epilogue(ok, 64, ok, None, 0, 0, None, 64, None, ok, 64, 1, rows, 64, 64, None, 0, None) == status
        assert L.gemm_bf16_epilogue_backward(ok, 64, ok, 64, ok, ok, 3, ok, ok, 1, ok, rows, 64, 64, ok, 1 << 40, None) == status


def test_workspace_sizes(L):
    # counters and whole FP32 tiles; none where one workgroup a tile fills the device
    assert L.fg8_gemm_bf16_workspace_bytes(8192, 8192, 8192) == 0
    assert (L.fg8_gemm_bf16_workspace_bytes(64, 2112, 7168) - 4096) % (64 * 64 * 4) == 0
    assert L.fg8_gemm_bf16_workspace_bytes(0, 64, 64) == 0 and L.fg8_gemm_bf16_backward_workspace_bytes(0, 64, 64) == 0
    # the backward pass keeps the counters' place and holds dz, odd widths rounded up
    assert L.fg8_gemm_bf16_backward_workspace_bytes(100, 33, 64) >= 4096 + 100 * 40 * 2
    assert L.fg8_layer_norm_backward_workspace_bytes(0, 64, 1) == 0
    assert L.fg8_layer_norm_backward_workspace_bytes(10, 64, 1) >= 10 * 2 * 64 * 4


def test_norm(L):
    def call(x=ok, ldx=64, xb=1, w=ok, b=None, wb=0, eps=1e-5, rows=4, cols=64, y=ok, mean=ok, rstd=ok):
        return L.layer_norm(x, ldx, xb, w, b, wb, eps, rows, cols, y, mean, rstd, None)
    for a in ({"x": None}, {"x": odd}, {"w": None}, {"b": odd}, {"y": None}, {"mean": None}, {"rstd": None}, {"xb": 2}, {"wb": -1},
              {"eps": -1.0}, {"eps": float("nan")}, {"rows": -1}, {"cols": 0}, {"ldx": 63}):
        assert call(**a) == EINVAL, a
    assert call(cols=32769, ldx=32769) == EUNSUPPORTED
    assert call(rows=0, x=None, y=None, mean=None, rstd=None) == OK

    def back(dy=ok, x=ok, w=ok, mean=ok, rstd=ok, rows=4, cols=64, dx=ok, dw=ok, db=ok, ws=ok, size=1 << 20, ld=64):
        return L.layer_norm_backward(dy, ld, x, ld, 1, w, 0, mean, rstd, rows, cols, dx, dw, db, ws, size, None)
    for a in ({"dy": None}, {"x": None}, {"w": None}, {"mean": None}, {"rstd": None}, {"dx": None}, {"dw": None}, {"db": None},
              {"ws": None}, {"ws": odd}, {"size": 100}, {"ld": 60}):
        assert back(**a) == EINVAL, a


def test_combine(L):
    def call(y=ok, b=1, rows=8, at=ok, p=ok, res=None, tokens=4, topk=2, hidden=64, out=ok):
        return L.moe_combine(y, b, rows, at, p, res, tokens, topk, hidden, out, None)
    for a in ({"y": None}, {"at": None}, {"p": odd}, {"res": odd}, {"out": None}, {"b": 2}, {"rows": 0}, {"tokens": -1},
              {"topk": 0}, {"topk": 257}, {"hidden": 0}):
        assert call(**a) == EINVAL, a
    assert call(hidden=60) == EUNSUPPORTED and call(tokens=1 << 31) == EUNSUPPORTED
    assert call(tokens=0, y=None, at=None, p=None, out=None) == OK

    def back(dout=ok, y=ok, rows=8, at=ok, owner=ok, p=ok, tokens=4, topk=2, hidden=64, dy=ok, dp=ok):
        return L.moe_combine_backward(dout, y, 1, rows, at, owner, p, tokens, topk, hidden, dy, dp, None)
    for a in ({"dout": None}, {"y": None}, {"at": None}, {"owner": None}, {"p": None}, {"dy": None}, {"dp": odd}):
        assert back(**a) == EINVAL, a
