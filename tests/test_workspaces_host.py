"""Where a call's workspace comes from, without a GPU: the library is a stand-in
that notes the workspace it is handed, tensors lie in host memory."""
import pytest
import torch

from moe_grouped_gemm_fp8_amd import _lib

SPLIT_BYTES = 4096 + 3 * 1024


class Library:
    """Takes any call, returns FG8_OK (or the size asked for) and notes the
    (pointer, bytes) of each product's workspace."""

    def __init__(self):
        self.given = []

    def fg8_gemm_workspace_bytes(self, m, n, k):
        return SPLIT_BYTES

    fg8_gemm_bf16_workspace_bytes = fg8_gemm_workspace_bytes

    def gemm_fp8_blockscaled(self, *args):
        ws = args[-3]
        self.given.append((getattr(ws, "value", ws), args[-2]))
        return 0

    gemm_bf16_epilogue = gemm_fp8_blockscaled


@pytest.fixture
def on_host(monkeypatch):
    library = Library()
    state = {"capturing": False}
    monkeypatch.setattr(_lib, "lib", lambda: library)
    monkeypatch.setattr(_lib, "_dev", lambda t, dtype, name: t)
    monkeypatch.setattr(_lib, "_rows", lambda t, dtype, name: t.shape[1])
    monkeypatch.setattr(_lib, "_stream_of", lambda t: 7)
    monkeypatch.setattr(_lib, "_stream", lambda: 7)
    monkeypatch.setattr(_lib, "_ws_cache", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: type("S", (), {"cuda_stream": 7}))
    return library, state


def _fp8_call():
    a, b = torch.zeros(64, 256, dtype=torch.uint8), torch.zeros(128, 256, dtype=torch.uint8)
    _lib.gemm_fp8_blockscaled(a, torch.zeros(2, 64), b, torch.zeros(1, 2))


def _bf16_call():
    _lib.gemm_bf16_epilogue(torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(128, 256, dtype=torch.bfloat16))


CALLS = {"fp8": _fp8_call, "bf16": _bf16_call}


@pytest.mark.parametrize("name", CALLS)
def test_a_recorded_call_leaves_nothing_in_the_cache(on_host, name):
    """Memory that a graph allocates, and clears only when it is replayed, must
    not reach a later eager call on the stream."""
    library, state = on_host
    state["capturing"] = True
    CALLS[name]()
    assert library.given[0][0] and library.given[0][1] >= SPLIT_BYTES
    assert not _lib._ws_cache


@pytest.mark.parametrize("name", CALLS)
def test_a_recorded_call_does_not_take_the_cached_workspace(on_host, name):
    """The cached buffer may be replaced by a larger one while the graph lives."""
    library, state = on_host
    CALLS[name]()
    state["capturing"] = True
    CALLS[name]()
    CALLS[name]()
    state["capturing"] = False
    CALLS[name]()
    eager, first, _, again = [p for p, _ in library.given]
    assert eager == again and first != eager
