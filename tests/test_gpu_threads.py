"""Calls of two host threads at once, on one stream: the same bits as alone.  Each
call below is several kernels that hand data on in the library's workspace."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _calls(fg8, dev, seed):
    g = torch.Generator(device=dev).manual_seed(seed)

    def bf16(*shape, scale=1.0):
        return (torch.randn(*shape, device=dev, generator=g) * scale).to(BF16)
    m, n, k, vocab = 40, 136, 1024, 900
    x, w, dh = bf16(m, k), bf16(2 * n, k, scale=k ** -0.5), bf16(m, n)
    h, z = fg8.gemm_bf16_gated(x, w, save_z=True)
    head = bf16(vocab, k, scale=k ** -0.5)
    t = torch.randint(0, vocab, (m,), device=dev, generator=g)
    dloss = torch.rand(m, device=dev, generator=g)

    def call():
        loss, lse = fg8.linear_cross_entropy(x, head, t)
        return (*fg8.gemm_bf16_gated_backward(dh, x, w, z, dw_dtype=torch.float32), loss, lse,
                *fg8.linear_cross_entropy_backward(dloss, x, head, t, lse))
    return call


def test_two_threads_on_one_stream(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    calls = [_calls(fg8, dev, seed) for seed in (1, 2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    start, got, failed = threading.Barrier(2), [[], []], []

    def work(i):
        try:
            start.wait(30)
            for _ in range(60):
                got[i].append(calls[i]())
        except Exception as e:      # (told below: an exception of a thread is no failure by itself)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for i in range(2):
        assert len(got[i]) == 60
        for turn in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(turn, want[i])), i
