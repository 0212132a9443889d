"""4-bit weights on the GPU: codes and scales bit for bit against the oracle, and
the products against float64.

Bounds of the products.  With integer x and scales of powers of two every partial
sum is an integer below 2^24 times one power of two: exact equality.  In general a
group's sum takes 2 GROUP products, (16 + code) x and -24 x, each exact, added in
FP32: every addition is off by at most 2^-23 (cut or rounded) of a partial sum that
T = sum of s (24 + 16 + code) |x| bounds; K / GROUP products with a scale, and
additions over groups, waves and the epilogue follow: e = (2 GROUP + 2 K / GROUP + 16)
2^-23 T.  An activation has a slope below 1.13 and is itself within 2^-19 of its
value; a BF16 output adds 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import int4, layer

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 4591 * k for i, k in enumerate(key)) + 3)


def _np(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------ quantize, dequantize
@pytest.mark.parametrize("scales", [F32, BF16])
@pytest.mark.parametrize("source", [F32, BF16])
@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (3, 64, 64), (33, 128, 128), (37, 544, 32), (64, 1024, 64),
                                             (100, 1664, 128), (5, 96, 32), (257, 512, 128)])
def test_quantize(dev, rows, cols, group, source, scales):
    print(f"int4 quantize {rows}x{cols} group {group} {source} {scales}", flush=True)
    g = _gen(1, rows, cols, group)
    w = torch.randn(2, rows, cols, generator=g) * torch.exp(3 * torch.randn(2, rows, 1, generator=g))
    w[0, 0, :group] = 0                                      # an all-zero group
    w[1, rows // 2, :8] = torch.tensor([7.0, 3.5, 2.5, -1.5, -0.5, 0.5, -7.0, 6.5]) * 2.0 ** 20       # ties
    w[1, rows // 2, 8:group] = 0
    w[0, -1, -group:] *= 2.0 ** -120                         # below the fast division's range
    w[1, -1, -group:] = w[1, -1, -group:].sign() * 2.0 ** -149   # a scale that underflows
    w = w.to(source)
    q, s = _fg8().int4_quantize(w.to(dev), group=group, scale_dtype=scales)
    assert q.shape == (2, rows, cols // 2) and s.shape == (2, cols // group, rows) and s.dtype == scales
    for b in range(2):
        codes, want = int4.quantize(w[b].float().numpy(), group, scales == BF16)
        assert np.array_equal(s[b].float().cpu().numpy(), want)
        assert np.array_equal(q[b].cpu().numpy(), int4.pack(codes))
        for out in (F32, BF16):
            back = _fg8().int4_dequantize(q, s, out_dtype=out)[b]          # (a slice need not be aligned)
            exact = torch.from_numpy(int4.values(codes, want)).float()     # code times scale: 24 + 4 bits, rounded once
            assert torch.equal(back.cpu(), exact.to(out))


def test_quantize_every_quotient(dev):
    """BF16 weights over many scales: quotients on and beside every border."""
    g = _gen(2)
    w = (torch.randint(-127, 128, (512, 1024), generator=g).float() * torch.randint(1, 200, (512, 1), generator=g)).to(BF16)
    q, s = _fg8().int4_quantize(w.to(dev), group=32)
    codes, want = int4.quantize(w.float().numpy(), 32)
    assert np.array_equal(s.cpu().numpy(), want) and np.array_equal(q.cpu().numpy(), int4.pack(codes))


def test_not_finite(dev):
    w = torch.randn(8, 256, generator=_gen(3))
    w[1, 5], w[2, 200], w[3, 0] = float("nan"), float("inf"), -float("inf")
    for scales in (F32, BF16):
        q, s = _fg8().int4_quantize(w.to(dev), group=64, scale_dtype=scales)
        v = _fg8().int4_dequantize(q, s, out_dtype=F32).cpu()
        lost = torch.zeros(8, 256, dtype=torch.bool)
        lost[1, :64] = lost[2, 192:] = lost[3, :64] = True
        assert torch.equal(v.isnan(), lost) and not v.isinf().any()


# ----------------------------------------------------------------- products
def _weights(g, sets, n, k, group, exact):
    """codes (0 among them) uint8 [sets, n, k], scales float32 [sets, k / group, n]"""
    codes = torch.randint(0, 16, (sets, n, k), generator=g, dtype=torch.uint8).numpy()
    if exact:
        scales = 2.0 ** torch.randint(-2, 3, (sets, k // group, n), generator=g).float()
    else:
        scales = (0.01 + torch.rand(sets, k // group, n, generator=g)).to(BF16).float() / 8
    return codes, scales


def _x(g, m, k, exact):
    return (torch.randint(-6, 7, (m, k), generator=g).float() if exact else torch.randn(m, k, generator=g)).to(BF16)


def _error(x, codes, scales):
    group = codes.shape[1] // scales.shape[0]
    t = np.abs(x) @ ((40.0 + codes) * np.repeat(np.asarray(scales, np.float64).T, group, 1)).T
    return (2 * group + 2 * codes.shape[1] / group + 16) * 2.0 ** -23 * t


def _check(got, want, err, what):
    g = _np(got)
    rounding = 2.0 ** -8 * (np.abs(want) + err) if got.dtype == BF16 else 0.0
    bad = ~(np.abs(g - want) <= err + rounding + 1e-38)
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} for {want[bad][0]}")


# m, n, k, group: single tokens, odd widths, every tile, partial chunks of k, several row blocks
DENSE = [(1, 1, 32, 32), (1, 16, 128, 128), (1, 33, 96, 32), (1, 100, 4224, 128), (2, 130, 192, 64), (5, 37, 2080, 32),
         (16, 64, 1024, 64), (17, 48, 160, 32), (31, 259, 384, 128), (33, 70, 2112, 64), (64, 36, 512, 128), (65, 52, 288, 32),
         (150, 20, 256, 128), (3, 8200, 128, 128), (4, 16400, 96, 32), (2, 4200, 288, 32), (3, 50, 160, 32), (4, 130, 4224, 128),
         (64, 4200, 288, 32)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("case", range(len(DENSE)))
def test_dense(dev, case, exact):
    m, n, k, group = DENSE[case]
    print(f"int4 {m}x{n}x{k} group {group} exact {exact}", flush=True)
    g = _gen(4, case, exact)
    codes, scales = _weights(g, 1, n, k, group, exact)
    x = _x(g, m, k, exact)
    codes, scales = codes[0], scales[0]
    want = _np(x) @ int4.values(codes, scales).T
    wide = torch.full((m, k + 8), float("nan"), dtype=BF16, device=dev)
    wide[:, :k] = x.to(dev)
    q = torch.from_numpy(int4.pack(codes)).to(dev)
    for dtype in (F32, BF16):
        y = _fg8().gemm_bf16_int4(wide[:, :k], q, scales.to(dtype).to(dev), out_dtype=F32)
        if exact:
            assert np.array_equal(_np(y), want), dtype
        else:
            _check(y, want, _error(_np(x), codes, scales), "y")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_epilogue(dev, act):
    m, n, k = 7, 77, 1184
    g = _gen(5, len(act))
    codes, scales = _weights(g, 1, n, k, 32, False)
    codes, scales, x = codes[0], scales[0] / 16, _x(g, m, k, False)
    bias, res = torch.randn(n, generator=g), torch.randn(m, n, generator=g).to(BF16)
    z = _np(x) @ int4.values(codes, scales).T + _np(bias)
    e = _error(_np(x), codes, scales) + 2.0 ** -23 * np.abs(z)
    want = layer.activation(act, z)
    e = 1.13 * e + 2.0 ** -19 * np.abs(want) + 2.0 ** -22 * (np.abs(want) + np.abs(_np(res)))
    buf = torch.full((m, n + 3), 5.0, dtype=BF16, device=dev)
    buf[:, :n] = res.to(dev)
    y = _fg8().gemm_bf16_int4(x.to(dev), torch.from_numpy(int4.pack(codes)).to(dev), scales.to(dev), bias.to(dev), buf[:, :n],
                              activation=act, out=buf[:, :n])      # onto the residual
    _check(y, want + _np(res), e, "y")
    assert (buf[:, n:] == 5).all()


# counts, rows before the first run, rows after the last, n, k, group
RUNS = [([1], 0, 0, 16, 32, 32), ([0, 0, 5], 0, 0, 37, 64, 64), ([3, 0, 17, 1], 2, 3, 72, 160, 32), ([64, 1, 65, 0, 63], 1, 0, 40, 384, 128),
        ([33, 20, 25], 0, 5, 66, 2176, 128), ([0] * 70 + [9] + [0] * 60 + [33], 0, 4, 20, 96, 32)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_runs(dev, case, gated):
    counts, before, after, n, k, group = RUNS[case]
    off = np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1]) + after
    print(f"int4 runs case {case} rows {rows} n {n} k {k} group {group} gated {gated}", flush=True)
    g = _gen(6, case)
    codes, scales = _weights(g, len(counts), 2 * n if gated else n, k, group, not gated)
    x = _x(g, rows, k, not gated)
    if gated:
        scales = scales / (k ** 0.5)
    w = np.stack([int4.values(c, s) for c, s in zip(codes, scales)])
    z, _ = layer.grouped(_np(x), w, off)
    x = x.to(dev)
    x[:before] = x[int(off[-1]):] = float("nan")
    y = _fg8().grouped_gemm_bf16_int4(x, torch.from_numpy(int4.pack(codes)).to(dev), scales.to(dev), torch.from_numpy(off).to(dev),
                                      activation="silu" if gated else "none", gated=gated, out_dtype=F32)
    if not gated:
        assert np.array_equal(_np(y), z)
        return
    xs, ez = np.nan_to_num(_np(x)), np.zeros_like(z)
    for e in range(len(counts)):
        ez[off[e]:off[e + 1]] = _error(xs[off[e]:off[e + 1]], codes[e], scales[e])
    a, u = np.abs(layer.activation("silu", z[:, :n])), np.abs(z[:, n:])
    _check(y, layer.gated("silu", z), 1.13 * ez[:, :n] * (u + ez[:, n:]) + a * ez[:, n:] + 2.0 ** -19 * a * u, "h")


@pytest.mark.parametrize("n,k,group", [(37, 64, 64), (21, 96, 32), (5, 384, 128), (40, 160, 32)])
def test_runs_bf16_scales(dev, n, k, group):
    """Experts whose scales start at odd elements, and a last one in no whole dword:
    exact, with poison behind the scales."""
    counts = [2, 0, 17, 1, 3]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    g = _gen(10, n, k)
    codes, scales = _weights(g, 5, n, k, group, True)
    x = _x(g, int(off[-1]), k, True)
    want, _ = layer.grouped(_np(x), np.stack([int4.values(c, s) for c, s in zip(codes, scales)]), off)
    room = torch.full((scales.numel() + 64,), float("nan"), dtype=BF16, device=dev)
    room[:scales.numel()] = scales.to(BF16).to(dev).flatten()
    y = _fg8().grouped_gemm_bf16_int4(x.to(dev), torch.from_numpy(int4.pack(codes)).to(dev), room[:scales.numel()].view(scales.shape),
                                      torch.from_numpy(off).to(dev), out_dtype=F32)
    assert np.array_equal(_np(y), want)


@pytest.mark.parametrize("m,n,k,group", [(1, 16, 128, 128), (1, 1031, 256, 32), (20, 45, 96, 32), (64, 128, 2304, 64)])
def test_gated_dense(dev, m, n, k, group):
    g = _gen(7, m, n)
    codes, scales = _weights(g, 1, 2 * n, k, group, False)
    codes, scales, x = codes[0], scales[0] / k ** 0.5, _x(g, m, k, False)
    z, ez = _np(x) @ int4.values(codes, scales).T, _error(_np(x), codes, scales)
    wide = torch.full((m, n + 4), 3.0, dtype=BF16, device=dev)
    y = _fg8().gemm_bf16_int4(x.to(dev), torch.from_numpy(int4.pack(codes)).to(dev), scales.to(dev), activation="gelu", gated=True,
                              out=wide[:, :n])
    a, u = np.abs(layer.activation("gelu", z[:, :n])), np.abs(z[:, n:])
    _check(y, layer.gated("gelu", z), 1.13 * ez[:, :n] * (u + ez[:, n:]) + a * ez[:, n:] + 2.0 ** -19 * (a + 2.0 ** -19) * u, "h")
    assert (wide[:, n:] == 3).all()


def test_block_in_four_bits(dev):
    """Quantize, gated product, second product onto the residual stream, against
    the BF16 products on the dequantized weights: the same sums of the same values
    but for the BF16 rounding of the weights, at most 2^-8 of each (and of h and
    y): 3 * 2^-8 of the sums of absolute values."""
    fg8, g = _fg8(), _gen(8)
    m, n, k = 3, 256, 512
    w1, w2 = torch.randn(2 * n, k, generator=g) * k ** -0.5, torch.randn(k, n, generator=g) * n ** -0.5
    x = torch.randn(m, k, generator=g).to(BF16).to(dev)
    q1, s1 = fg8.int4_quantize(w1.to(dev), group=64)
    q2, s2 = fg8.int4_quantize(w2.to(BF16).to(dev), group=128, scale_dtype=BF16)
    y = fg8.gemm_bf16_int4(fg8.gemm_bf16_int4(x, q1, s1, activation="silu", gated=True), q2, s2, residual=x)
    h = fg8.gemm_bf16_gated(x, fg8.int4_dequantize(q1, s1))
    want = fg8.gemm_bf16_epilogue(h, fg8.int4_dequantize(q2, s2), residual=x)
    z1 = np.abs(_np(x)) @ np.abs(_np(fg8.int4_dequantize(q1, s1))).T
    size = (z1[:, :n] * z1[:, n:]) @ np.abs(_np(fg8.int4_dequantize(q2, s2))).T + np.abs(_np(x))
    assert (np.abs(_np(y) - _np(want)) <= 3 * 2.0 ** -8 * size).all()


def test_captured(dev):
    fg8, g = _fg8(), _gen(9)
    codes, scales = _weights(g, 1, 200, 2048, 128, True)
    q, s, x = torch.from_numpy(int4.pack(codes[0])).to(dev), scales[0].to(dev), _x(g, 4, 2048, True).to(dev)
    want = fg8.gemm_bf16_int4(x, q, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fg8.gemm_bf16_int4(x, q, s)
    for i in range(4):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want), i
        assert torch.equal(fg8.gemm_bf16_int4(x, q, s), want)
