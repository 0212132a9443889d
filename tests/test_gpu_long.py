"""The BF16 operators on tensors of more than 2^31 elements, whose offsets do
not fit 32 bits.

Operands are small integers, so every FP32 sum here is exact in any order (all
stay below 2^24) and results are compared for equality: rows on both sides of
the element 2^31 and at the end against float64, or, where an operator rounds,
against the same operator on those rows alone.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROWS, COLS = 300_000, 7200      # 2.16e9 elements


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _ints(g, most, *shape):
    """Integers of [-most, most] in BF16."""
    return torch.randint(-most, most + 1, shape, generator=g, device=g.device, dtype=torch.int8).to(BF16)


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _samples(cols):
    """Rows at the start, around element 2^31 and at the end."""
    edge = 2 ** 31 // cols
    return torch.tensor([*range(6), *range(edge - 3, edge + 4), *range(ROWS - 6, ROWS)])


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def test_grouped_long_rows(dev):
    fg8, g = _fg8(), _gen(dev, 1)
    x, w = _ints(g, 1, ROWS, COLS), _ints(g, 1, 3, 72, COLS)
    off = torch.tensor([4, 9, 298_265, ROWS - 3], dtype=I32, device=dev)
    y = fg8.grouped_gemm_bf16(x, w, off, out_dtype=F32)
    expert = torch.bucketize(torch.arange(ROWS, device=dev), off.long(), right=True) - 1
    for r in _samples(COLS).tolist():
        e = int(expert[r])
        want = x[r].double() @ w[e].double().T.contiguous() if 0 <= e < 3 else torch.zeros(72, device=dev)
        assert torch.equal(y[r].double(), want.double()), f"row {r}"
    del y
    dx = fg8.grouped_gemm_bf16_dgrad(x[:, :72].contiguous(), w, off)     # dx is the long one
    for r in _samples(COLS).tolist():
        e = int(expert[r])
        want = x[r, :72].double() @ w[e].double() if 0 <= e < 3 else torch.zeros(COLS, device=dev)
        assert torch.equal(dx[r].double(), want.double()), f"row {r}"
    del dx
    dw = fg8.grouped_gemm_bf16_wgrad(_strip(x), x, off)
    for e in range(3):
        want = torch.zeros(8, COLS, dtype=torch.float64, device=dev)
        for a in range(int(off[e]), int(off[e + 1]), 20_000):
            b = min(a + 20_000, int(off[e + 1]))
            want += x[a:b, :8].double().T.contiguous() @ x[a:b].double()
        assert torch.equal(dw[e].double(), want), f"expert {e}"


def _strip(x):
    return x[:, :8]                # (strided rows)


def test_grouped_many_weights(dev):
    fg8, g = _fg8(), _gen(dev, 2)
    E, n, k, per = 260, 4096, 2048, 3                        # 2.18e9 weights
    off = (torch.arange(E + 1, device=dev) * per).to(I32)
    x, dy = _ints(g, 1, E * per, k), _ints(g, 1, E * per, n)
    for dtype in (F32, BF16):
        dw = fg8.grouped_gemm_bf16_wgrad(dy, x, off, out_dtype=dtype)
        for e in (0, 1, 254, 255, 256, 257, 259):
            at = slice(e * per, (e + 1) * per)
            assert torch.equal(dw[e].double(), dy[at].double().T.contiguous() @ x[at].double()), f"expert {e}"
        if dtype == F32:
            del dw
    y = fg8.grouped_gemm_bf16(x, dw, off, out_dtype=F32)
    dx = fg8.grouped_gemm_bf16_dgrad(dy, dw, off, out_dtype=F32)
    for e in (0, 1, 254, 255, 256, 257, 259):
        at = slice(e * per, (e + 1) * per)
        assert torch.equal(y[at].double(), x[at].double() @ dw[e].double().T.contiguous()), f"expert {e}"
        assert torch.equal(dx[at].double(), dy[at].double() @ dw[e].double()), f"expert {e}"


def test_dense_long_output(dev):
    fg8, g = _fg8(), _gen(dev, 3)
    x, w, b = _ints(g, 2, ROWS, 8), _ints(g, 2, COLS, 8), _ints(g, 3, COLS)
    res = _ints(g, 3, ROWS, COLS)
    y, z = fg8.gemm_bf16_epilogue(x, w, bias=b, residual=res, activation="relu", save_z=True)
    at = _samples(COLS).to(dev)
    want = x[at].double() @ w.double().T.contiguous() + b.double()
    assert torch.equal(z[at].double(), want)
    assert torch.equal(y[at].double(), want.clamp(min=0) + res[at].double())
    del y
    dx, dw, db = fg8.gemm_bf16_epilogue_backward(res, x, w, z=z, activation="relu", dw_dtype=F32)
    dz = res[at].double() * (z[at] > 0)
    assert torch.equal(dx[at], (dz @ w.double()).to(BF16))
    want_w, want_b = torch.zeros(COLS, 8, dtype=torch.float64, device=dev), torch.zeros(COLS, dtype=torch.float64, device=dev)
    for a in range(0, ROWS, 20_000):
        dz = res[a:a + 20_000].double() * (z[a:a + 20_000] > 0)
        want_w += dz.T.contiguous() @ x[a:a + 20_000].double()
        want_b += dz.sum(0)
    assert torch.equal(dw.double(), want_w) and torch.equal(db.double(), want_b)


def test_layer_norm_long(dev):
    fg8, g = _fg8(), _gen(dev, 4)
    x, dy = _ints(g, 4, ROWS, COLS), _ints(g, 4, ROWS, COLS)
    w, b = torch.rand(COLS, generator=g, device=dev), torch.rand(COLS, generator=g, device=dev)
    at = _samples(COLS).to(dev)
    y, mean, rstd = fg8.layer_norm(x, w, b)
    part = fg8.layer_norm(x[at], w, b)
    assert torch.equal(y[at], part[0]) and torch.equal(mean[at], part[1]) and torch.equal(rstd[at], part[2])
    del y
    dx, dw, db = fg8.layer_norm_backward(dy, x, w, mean, rstd)
    assert torch.equal(dx[at], fg8.layer_norm_backward(dy[at], x[at], w, mean[at], rstd[at])[0])
    want = torch.zeros(COLS, dtype=torch.float64, device=dev)
    for a in range(0, ROWS, 20_000):
        want += dy[a:a + 20_000].double().sum(0)
    assert torch.equal(db.double(), want)


def test_combine_long(dev):
    fg8, g = _fg8(), _gen(dev, 5)
    y = _ints(g, 2, ROWS, COLS)
    held = _samples(COLS)[:18]
    token_row = held.to(I32).reshape(9, 2).to(dev)
    row_token = torch.full((ROWS,), -1, dtype=I32)
    row_token[held] = (torch.arange(18) // 2).to(I32)
    p = 2.0 ** torch.randint(-2, 3, (9, 2), generator=g, device=dev).float()
    out = fg8.moe_combine(y, token_row, p)
    rows = y[held.to(dev)].double().reshape(9, 2, COLS)
    assert torch.equal(out.double(), (rows * p.double()[..., None]).sum(1))
    dout = _ints(g, 2, 9, COLS)
    dy, dp = fg8.moe_combine_backward(dout, y, token_row, row_token.to(dev), p)
    assert torch.equal(dy[held.to(dev)].double().reshape(9, 2, COLS), p.double()[..., None] * dout.double()[:, None])
    assert torch.equal(dp.double(), (rows * dout.double()[:, None]).sum(2))
    dy[held.to(dev)] = 0
    assert not any(bool(dy[a:a + 50_000].any()) for a in range(0, ROWS, 50_000))
