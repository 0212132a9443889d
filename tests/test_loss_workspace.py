"""The workspace of the loss's backward pass: what a call without a weight gradient
asks for.  Without a GPU call: refused before any launch, and the Python layer with
a library that notes what it is asked for."""
import ctypes
import re

import pytest
import torch

from moe_grouped_gemm_fp8_amd import _lib

P = ctypes.c_void_p
ok = P(0x10000)      # never dereferenced: nothing here is launched


@pytest.mark.parametrize("m,vocab,k", [(40, 1000, 64), (80, 72, 64), (8192, 32769, 64)])
def test_without_a_weight_gradient_its_type_does_not_matter(m, vocab, k):
    L = _lib.lib()
    size = L.fg8_linear_cross_entropy_backward_workspace_bytes
    assert size(m, vocab, k, _lib.OUT_F32) > size(m, vocab, k, _lib.OUT_BF16)
    for dw, out in ((None, _lib.OUT_F32), (None, _lib.OUT_BF16), (ok, _lib.OUT_F32), (ok, _lib.OUT_BF16)):
        need = size(m, vocab, k, out if dw else _lib.OUT_BF16)
        assert L.linear_cross_entropy_backward(ok, ok, k, ok, ok, 0, ok, ok, dw, out, m, vocab, k, ok, need - 1, None) == 1
        said = int(re.search(rb"workspace of (\d+) bytes", L.fg8_last_error()).group(1))
        assert said == need, (dw, out)


@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
def test_the_python_layer_asks_for_what_is_wanted(monkeypatch, needs, dw_dtype):
    asked, given = [], []

    class Library:
        def fg8_linear_cross_entropy_backward_workspace_bytes(self, m, vocab, k, out):
            asked.append(out)
            return 8192

        def linear_cross_entropy_backward(self, *args):
            given.append(args)
            return 0
    monkeypatch.setattr(_lib, "lib", Library)
    monkeypatch.setattr(_lib, "_dev", lambda t, dtype, name: t)
    monkeypatch.setattr(_lib, "_rows", lambda t, dtype, name: t.shape[1])
    monkeypatch.setattr(_lib, "_stream_of", lambda t: 7)
    monkeypatch.setattr(_lib, "_ws_cache", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.bfloat16)
    dx, dw = _lib.linear_cross_entropy_backward(torch.zeros(4), x, w, torch.zeros(4, dtype=torch.int64), torch.zeros(4),
                                                dw_dtype=dw_dtype, needs=needs)
    assert (dx is not None, dw is not None) == needs
    two_parts = needs[1] and dw_dtype == torch.float32
    assert asked == [_lib.OUT_F32 if two_parts else _lib.OUT_BF16] and len(given) == 1
