"""The gated BF16 products without a GPU: refusals that come before any launch,
and the calls on nothing."""
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


def test_forward(L):
    need = L.fg8_gemm_bf16_gated_workspace_bytes(40, 264, 7168)
    assert need > 4096

    def call(x=ok, ldx=7168, w=ok, act=2, z=None, h=ok, ldh=264, out=1, m=40, n=264, k=7168, ws=ok, size=need):
        return L.gemm_bf16_gated(x, ldx, w, act, z, h, ldh, out, m, n, k, ws, size, None)
    for a in ({"x": None}, {"w": odd}, {"h": None}, {"z": odd}, {"act": 4}, {"act": -1}, {"m": -1}, {"n": 0}, {"k": 0}, {"ldh": 263},
              {"ldx": 7160}, {"ldx": 7172}, {"out": 2}, {"ws": None}, {"ws": odd}, {"size": need - 1}, {"m": 1 << 31}):
        assert call(**a) == EINVAL, a
    for a in ({"k": 7164}, {"n": (1 << 21) + 1, "ldh": 1 << 22}, {"k": (1 << 22) + 8, "ldx": (1 << 22) + 8}, {"m": (1 << 31) - 1000}):
        assert call(**a) == EUNSUPPORTED, a
    assert call(m=0, x=None, w=None, h=None) == OK

    def runs(x=ok, ldx=64, w=ok, off=ok, act=2, z=None, h=ok, ldh=64, out=1, rows=10, n=64, k=64, e=4):
        return L.grouped_gemm_bf16_gated(x, ldx, w, off, act, z, h, ldh, out, rows, n, k, e, None)
    for a in ({"x": odd}, {"w": None}, {"off": None}, {"h": odd}, {"z": odd}, {"act": 7}, {"rows": -1}, {"e": 0}, {"e": 1025}, {"ldh": 60},
              {"ldx": 60}, {"out": -1}):
        assert runs(**a) == EINVAL, a
    assert runs(k=60) == EUNSUPPORTED and runs(n=1 << 22, ldh=1 << 22) == EUNSUPPORTED
    assert runs(rows=0, x=None, w=None, h=None) == OK


def test_backward(L):
    def call(dh=ok, lddh=64, x=ok, ldx=64, w=ok, z=ok, act=3, dx=ok, dw=ok, out=1, m=8, n=64, k=64, ws=ok, size=1 << 30):
        return L.gemm_bf16_gated_backward(dh, lddh, x, ldx, w, z, act, dx, dw, out, m, n, k, ws, size, None)

    def runs(dh=ok, lddh=64, x=ok, ldx=64, w=ok, z=ok, off=ok, act=3, dx=ok, dw=ok, out=1, m=8, n=64, k=64, e=4, ws=ok, size=1 << 30):
        return L.grouped_gemm_bf16_gated_backward(dh, lddh, x, ldx, w, z, off, act, dx, dw, out, m, n, k, e, ws, size, None)
    for f, e in ((call, 0), (runs, 4)):
        need = L.fg8_gemm_bf16_gated_backward_workspace_bytes(8, 64, 64, e)
        assert need == 4096 + 8 * 128 * 2 or e == 0
        for a in ({"dh": None}, {"z": None}, {"w": None}, {"x": None}, {"dx": None, "dw": None}, {"dx": odd}, {"dw": odd}, {"act": 9},
                  {"m": 0}, {"ws": None}, {"size": need - 1}, {"lddh": 63}, {"ldx": 60}, {"out": 5}):
            assert f(**a) == EINVAL, a
        assert f(k=60) == EUNSUPPORTED
    assert runs(off=None) == EINVAL and runs(e=0) == EINVAL
    # odd widths: dz's rows are whole 16-byte pieces
    assert L.fg8_gemm_bf16_gated_backward_workspace_bytes(3, 5, 64, 1) == 4096 + 3 * 16 * 2
    assert L.fg8_gemm_bf16_gated_backward_workspace_bytes(0, 5, 64, 1) == 0


def test_python_layer_refuses():
    import moe_grouped_gemm_fp8_amd as fg8
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):            # not on the GPU
        fg8.gemm_bf16_gated(x, w)
    with pytest.raises(KeyError):
        fg8.gemm_bf16_gated(x, w, activation="tanh")
