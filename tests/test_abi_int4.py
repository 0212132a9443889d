"""The 4-bit weights without a GPU: refusals that come before any launch, and the
calls on nothing."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED = 0, 1, 2
ok, odd = P(0x10000), P(0x10008)      # never dereferenced: nothing here is launched


@pytest.fixture(scope="module")
def L():
    from moe_grouped_gemm_fp8_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libfg8.so is not built (run __graft_entry__.build())")
    return _lib.lib()


def test_quantize(L):
    def quantize(w=ok, bf=1, batch=1, rows=4, cols=256, group=128, q=ok, s=ok, sbf=0):
        return L.int4_quantize(w, bf, batch, rows, cols, group, q, s, sbf, None)

    def dequantize(w=ok, bf=1, batch=1, rows=4, cols=256, group=128, q=ok, s=ok, sbf=0):
        return L.int4_dequantize(q, s, sbf, batch, rows, cols, group, w, bf, None)
    for f in (quantize, dequantize):
        for a in ({"w": None}, {"w": odd}, {"q": odd}, {"q": None}, {"s": None}, {"s": odd}, {"bf": 2}, {"sbf": 2}, {"batch": 0},
                  {"batch": 65536}, {"rows": 0}, {"cols": 0}, {"rows": -1}):
            assert f(**a) == EINVAL, (f, a)
        for a in ({"group": 16}, {"group": 256}, {"group": 0}, {"cols": 192}, {"cols": 255}, {"rows": (1 << 22) + 1},
                  {"cols": (1 << 22) + 128}, {"batch": 4096, "rows": 1 << 22, "cols": 4096}):
            assert f(**a) == EUNSUPPORTED, (f, a)


def test_products(L):
    def dense(x=ok, ldx=256, q=ok, s=ok, sbf=0, group=64, bias=None, bb=0, act=2, gated=0, res=None, ldr=40, y=ok, ldy=40, out=1, m=3,
              n=40, k=256):
        return L.gemm_bf16_int4(x, ldx, q, s, sbf, group, bias, bb, act, gated, res, ldr, y, ldy, out, m, n, k, None)

    def runs(x=ok, ldx=256, q=ok, s=ok, sbf=0, group=64, off=ok, act=2, gated=0, y=ok, ldy=40, out=1, m=3, n=40, k=256, e=2):
        return L.grouped_gemm_bf16_int4(x, ldx, q, s, sbf, group, off, act, gated, y, ldy, out, m, n, k, e, None)
    for f in (dense, runs):
        for a in ({"x": None}, {"x": odd}, {"q": None}, {"q": odd}, {"s": None}, {"s": odd}, {"y": None}, {"sbf": 3}, {"act": 4}, {"act": -1},
                  {"gated": 2}, {"out": 2}, {"m": -1}, {"m": 1 << 31}, {"n": 0}, {"k": 0}, {"ldx": 248}, {"ldx": 260}, {"ldy": 39}):
            assert f(**a) == EINVAL, (f, a)
        for a in ({"group": 48}, {"k": 224}, {"n": (1 << 22) + 1, "ldy": 1 << 22}, {"gated": 1, "n": (1 << 21) + 8, "ldy": 1 << 22},
                  {"m": (1 << 31) - 1}, {"ldx": (1 << 22) + 8}):
            assert f(**a) == EUNSUPPORTED, (f, a)
        assert f(m=0, x=None, q=None, s=None, y=None) == OK
    for a in ({"bias": odd}, {"bb": 2}, {"res": odd}, {"res": ok, "ldr": 39}, {"gated": 1, "bias": ok}, {"gated": 1, "res": ok}):
        assert dense(**a) == EINVAL, a
    assert runs(off=None) == EINVAL and runs(e=0) == EINVAL and runs(e=1025) == EINVAL
    # more tiles than a launch holds
    assert dense(m=(1 << 31) - 1024, n=1 << 22, ldy=1 << 22) == EUNSUPPORTED
    assert b"launch" in L.fg8_last_error()


def test_python_layer_refuses():
    import moe_grouped_gemm_fp8_amd as fg8
    w = torch.zeros(16, 64)
    with pytest.raises(ValueError):            # not on the GPU
        fg8.int4_quantize(w, group=32)
    with pytest.raises(ValueError):
        fg8.gemm_bf16_int4(w.to(torch.bfloat16), torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(2, 16))
