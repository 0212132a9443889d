"""Refusals of the Python layer that come before the library is called, without
a GPU: tensors in host memory that say they are on a device.  The library is a
stand-in that must not be reached."""
import pytest
import torch

from moe_grouped_gemm_fp8_amd import _lib

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class OnDevice(torch.Tensor):
    """Host memory that claims to lie on device `index`."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def gpu(*shape, dtype=BF16, index=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


class Unreached:
    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 8192
        raise AssertionError(f"{name} was called")


@pytest.fixture(autouse=True)
def stand_in(monkeypatch):
    monkeypatch.setattr(_lib, "lib", lambda: Unreached())
    monkeypatch.setattr(_lib, "_stream_of", lambda t: 7)
    monkeypatch.setattr(_lib, "_stream", lambda: 7)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)


PRODUCTS = {
    "fp8": lambda **kw: _lib.gemm_fp8_blockscaled(gpu(64, 256, dtype=U8), gpu(2, 64, dtype=F32), gpu(128, 256, dtype=U8),
                                                  gpu(1, 2, dtype=F32), out=gpu(64, 128), **kw),
    "forward": lambda **kw: _lib.gemm_bf16_epilogue(gpu(64, 256), gpu(128, 256), out=gpu(64, 128), **kw),
    "backward": lambda **kw: _lib.gemm_bf16_epilogue_backward(gpu(64, 128), gpu(64, 256), gpu(128, 256), **kw),
}


@pytest.mark.parametrize("name", PRODUCTS)
def test_a_workspace_that_the_gpu_cannot_use_is_refused(name):
    with pytest.raises(ValueError, match="workspace must be a CUDA"):
        PRODUCTS[name](workspace=torch.zeros(1 << 20, dtype=U8))
    # its elements would reach past its memory
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        PRODUCTS[name](workspace=gpu(1 << 10, 64, dtype=U8)[:, :32])
