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
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


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


# Each call with its tensor operands; every one of them in turn lies on another
# device than the current one.
def _call(fn, operands, **kw):
    return fn, operands, kw


def _calls():
    e, k = 2, 256
    rows, w, off = gpu(64, k), gpu(e, 128, k), gpu(e + 1, dtype=I32)
    token_row, weights = gpu(8, 2, dtype=I32), gpu(8, 2, dtype=F32)
    vec, stat = gpu(k, dtype=F32), gpu(64, dtype=F32)
    return {
        "quantize": _call(_lib.fp8_quantize, [rows]),
        "fp8": _call(_lib.gemm_fp8_blockscaled, [gpu(64, k, dtype=U8), gpu(2, 64, dtype=F32), gpu(128, k, dtype=U8), gpu(1, 2, dtype=F32)],
                     out=gpu(64, 128)),
        "layout": _call(_lib.moe_contiguous_layout_fp8, [rows, gpu(64, 2, dtype=I32)], num_experts=4),
        "grouped": _call(_lib.grouped_gemm_bf16, [rows, w, off]),
        "dgrad": _call(_lib.grouped_gemm_bf16_dgrad, [gpu(64, 128), w, off]),
        "wgrad": _call(_lib.grouped_gemm_bf16_wgrad, [gpu(64, 128), rows, off]),
        "dense": _call(_lib.gemm_bf16_epilogue, [rows, gpu(128, k), gpu(128, dtype=F32), gpu(64, 128)]),
        "dense backward": _call(_lib.gemm_bf16_epilogue_backward, [gpu(64, 128), rows, gpu(128, k), gpu(64, 128)], activation="silu"),
        "norm": _call(_lib.layer_norm, [rows, vec, gpu(k, dtype=F32)]),
        "norm backward": _call(_lib.layer_norm_backward, [gpu(64, k), rows, vec, stat, gpu(64, dtype=F32)]),
        "combine": _call(_lib.moe_combine, [rows, token_row, weights, gpu(8, k)]),
        "combine backward": _call(_lib.moe_combine_backward, [gpu(8, k), rows, token_row, gpu(64, dtype=I32), weights]),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_operands_on_another_device_are_refused(name):
    fn, operands, kw = _calls()[name]
    with pytest.raises(AssertionError, match="was called"):      # all on the current device: on to the library
        fn(*operands, **kw)
    for t in operands:
        t.index = 1
        with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
            fn(*operands, **kw)
        t.index = 0
