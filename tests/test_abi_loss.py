"""The cross entropy of a linear head without a GPU: refusals that come before any
launch, and the calls on nothing."""
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
    need = L.fg8_linear_cross_entropy_workspace_bytes(40, 1000, 64)
    # counters, target logits, a maximum and a sum for each row and 128 classes
    assert need == 4096 + 160 + 8 * 40 * 8
    # with a long k partial tiles of 64 x 128 besides
    longer = L.fg8_linear_cross_entropy_workspace_bytes(40, 1000, 4096)
    assert longer > need and (longer - need) % (64 * 128 * 4) == 0
    assert L.fg8_linear_cross_entropy_workspace_bytes(0, 1000, 64) == 0

    def call(x=ok, ldx=64, w=ok, t=ok, wide=1, loss=ok, lse=ok, m=40, v=1000, k=64, ws=ok, size=need):
        return L.linear_cross_entropy(x, ldx, w, t, wide, loss, lse, m, v, k, ws, size, None)
    for a in ({"x": None}, {"x": odd}, {"w": None}, {"t": None}, {"t": odd}, {"loss": None}, {"lse": odd}, {"wide": 2}, {"m": -1}, {"v": 0},
              {"k": 0}, {"ldx": 56}, {"ldx": 68}, {"ws": None}, {"ws": odd}, {"size": need - 1}, {"m": 1 << 31}):
        assert call(**a) == EINVAL, a
    for a in ({"k": 60}, {"v": (1 << 22) + 1}, {"k": (1 << 22) + 8, "ldx": (1 << 22) + 8}, {"m": (1 << 31) - 1}, {"ldx": (1 << 22) + 8}):
        assert call(**a) == EUNSUPPORTED, a
    assert call(m=0, x=None, w=None, t=None, loss=None, lse=None, ws=None) == OK


def test_backward(L):
    size = L.fg8_linear_cross_entropy_backward_workspace_bytes
    need = size(40, 1000, 64, 1)
    # what dlogits' rounding left, and x twice where there are no more rows than classes
    assert size(40, 1000, 64, 0) == need + 40 * 1000 * 2 + 2 * 40 * 64 * 2
    assert size(80, 72, 64, 0) == size(80, 72, 64, 1) + 80 * 72 * 2
    # one piece of the vocabulary while its dlogits are 512 MB at most, then pieces of
    # one size in units of 8192 classes, and dx's sums
    one, two = size(8192, 32768, 64, 1), size(8192, 32769, 64, 1)
    assert one >= (512 << 20) + 4096 and (384 << 20) + 8192 * 64 * 4 < two < one

    def call(d=ok, x=ok, ldx=64, w=ok, t=ok, wide=0, lse=ok, dx=ok, dw=ok, out=1, m=40, v=1000, k=64, ws=ok, n=need):
        return L.linear_cross_entropy_backward(d, x, ldx, w, t, wide, lse, dx, dw, out, m, v, k, ws, n, None)
    for a in ({"d": None}, {"x": odd}, {"w": None}, {"t": None}, {"lse": None}, {"dx": odd}, {"dw": odd}, {"dx": None, "dw": None},
              {"wide": -1}, {"out": 2}, {"m": 0}, {"v": 0}, {"ldx": 48}, {"ws": None}, {"n": need - 1}, {"out": 0}):
        assert call(**a) == EINVAL, a
    assert call(k=60) == EUNSUPPORTED and call(v=(1 << 22) + 1) == EUNSUPPORTED


def test_python_layer_refuses():
    import moe_grouped_gemm_fp8_amd as fg8
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):            # not on the GPU
        fg8.linear_cross_entropy(x, w, torch.zeros(4, dtype=torch.int64))
