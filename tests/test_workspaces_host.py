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


# ------------------------------------------------------------- what is kept
class Operand:
    """Allocates like a tensor and notes what the cache held meanwhile."""

    def __init__(self):
        self.device, self.held = torch.device("cpu"), []

    def new_empty(self, nbytes, dtype):
        self.held.append(sum(w.numel() for w in _lib._ws_cache.values()))
        return torch.full((nbytes,), 7, dtype=dtype)


def test_a_large_workspace_is_not_kept(on_host):
    """16384 x 16384: dz alone is half a gigabyte."""
    t, most = Operand(), _lib.WS_KEEP_BYTES
    small = _lib._workspace_of(1 << 20, t, 7)[0]
    big, ptr, size = _lib._workspace_of(most + 16, t, 7)
    assert size == most + 16 and ptr == big.data_ptr() and not big[:_lib.WS_COUNTER_BYTES].any()
    assert _lib._workspace_of(1 << 20, t, 7)[0] is small
    assert sum(w.numel() for w in _lib._ws_cache.values()) == 1 << 20


def test_a_growing_workspace_clears_its_counters_and_frees_the_old_one(on_host):
    t = Operand()
    first = _lib._workspace_of(1 << 16, t, 7)[0]
    assert not first[:_lib.WS_COUNTER_BYTES].any()
    del first
    second = _lib._workspace_of(1 << 18, t, 7)[0]
    assert t.held == [0, 0], "the old buffer was held while the new one was allocated"
    assert not second[:_lib.WS_COUNTER_BYTES].any() and bool((second[_lib.WS_COUNTER_BYTES:] == 7).all())


def test_the_counters_are_the_kernels():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "moe_grouped_gemm_fp8_amd", "csrc", "fg8_internal.h")).read()
    tiles = int(re.search(r"kSplitKMaxTiles = (\d+);", text).group(1))
    assert "kSplitKCounterBytes = kSplitKMaxTiles * sizeof(int32_t);" in text
    assert _lib.WS_COUNTER_BYTES == 4 * tiles
    # the kept size holds every split product of the device
    L = _lib.lib()
    most = 0
    for m in (1, 16, 33, 64, 128, 200, 256, 300, 384, 512, 700, 1024):
        for n in (64, 512, 1024, 2112, 4096, 7168):
            most = max(most, L.fg8_gemm_bf16_workspace_bytes(m, n, 8192), L.fg8_gemm_workspace_bytes(m, n, 8192))
    assert most <= _lib.WS_KEEP_BYTES
