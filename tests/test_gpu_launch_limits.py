"""The largest launches that the argument checks let through run: the MoE
combine at 2^24 - 1 workgroups of 256 threads, with few columns.  Values are
small integers, so every result is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
MOST = (2 ** 32 - 1) // 256


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def test_combine_of_the_most_tokens(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    tokens, rows = 4 * MOST, 1000
    y = (torch.arange(rows * 8, device=dev).reshape(rows, 8) % 201 - 100).to(BF16)
    at = (torch.arange(tokens, device=dev) % (rows + 1)).to(I32).reshape(tokens, 1)      # row `rows` adds nothing
    out = fg8.moe_combine(y, at, torch.full((tokens, 1), 2.0, device=dev))
    table = torch.cat([2 * y, torch.zeros(1, 8, dtype=BF16, device=dev)])
    for a in range(0, tokens, 1 << 24):
        assert torch.equal(out[a:a + (1 << 24)], table[at[a:a + (1 << 24), 0].long()]), f"tokens from {a}"
    with pytest.raises(fg8.Fg8Error, match="exceed a launch"):
        fg8.moe_combine(y, torch.zeros(tokens + 1, 1, dtype=I32, device=dev), torch.zeros(tokens + 1, 1, device=dev))


def test_combine_backward_of_the_most_tokens(dev):
    import moe_grouped_gemm_fp8_amd as fg8
    tokens, rows = MOST - 250, 1000
    y = (torch.arange(rows * 8, device=dev).reshape(rows, 8) % 5 - 2).to(BF16)
    dout = (torch.arange(tokens * 8, device=dev).reshape(tokens, 8) % 7 - 3).to(BF16)
    # the last 999 tokens have a row each, row 7 has none
    at = torch.full((tokens, 1), -1, dtype=I32, device=dev)
    owner = torch.full((rows,), -1, dtype=I32, device=dev)
    held = torch.tensor([r for r in range(rows) if r != 7], dtype=I32, device=dev)
    at[tokens - 999:, 0] = held
    owner[held.long()] = torch.arange(tokens - 999, tokens, dtype=I32, device=dev)
    dy, dp = fg8.moe_combine_backward(dout, y, at, owner, torch.full((tokens, 1), 2.0, device=dev))
    assert torch.equal(dy[held.long()], 2 * dout[tokens - 999:]) and not dy[7].any()
    assert torch.equal(dp[tokens - 999:, 0], (dout[tokens - 999:].float() * y[held.long()].float()).sum(1))
    assert not dp[:tokens - 999].any()
