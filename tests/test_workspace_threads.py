"""Two host threads on one stream: a call of several kernels keeps data in its
workspace between them, so the threads' calls must not share one.  Without a GPU:
tensors lie in host memory."""
import threading

import pytest
import torch

from moe_grouped_gemm_fp8_amd import _lib


@pytest.fixture
def cache(monkeypatch):
    kept = {}
    monkeypatch.setattr(_lib, "_ws_cache", kept)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return kept


def _in_thread(f):
    got = []
    t = threading.Thread(target=lambda: got.append(f()))
    t.start()
    t.join()
    return got[0]


def test_each_thread_has_its_own(cache):
    t = torch.zeros(1)
    mine = _lib._workspace_of(1 << 16, t, 7)[0]
    ready, done, got = threading.Barrier(3), threading.Barrier(3), {}

    def call(name):
        ready.wait(30)
        got[name] = [_lib._workspace_of(1 << 16, t, 7)[0] for _ in range(3)]
        done.wait(30)
    threads = [threading.Thread(target=call, args=(n,)) for n in "ab"]
    for th in threads:
        th.start()
    ready.wait(30)
    done.wait(30)
    for th in threads:
        th.join()
    assert all(w is got[n][0] for n in "ab" for w in got[n])
    assert len({w.data_ptr() for w in (mine, got["a"][0], got["b"][0])}) == 3
    assert _lib._workspace_of(1 << 16, t, 7)[0] is mine


def test_what_ended_threads_kept_is_given_back(cache):
    t = torch.zeros(1)
    mine = _lib._workspace_of(1 << 16, t, 7)[0]
    for _ in range(5):
        _in_thread(lambda: _lib._workspace_of(1 << 16, t, 7)[1])
    _lib._workspace_of(1 << 16, t, 8)
    assert len(cache) <= 3 and any(w is mine for w in cache.values())
