"""Every tile of the BF16 products at a size that is given it, the choice
asserted: a changed rule cannot leave an instance of the kernels untested.

References are float64 products on the GPU.  Bounds, with u = 2^-24: a sum of K
products of BF16 values is off by at most 2 (K + 1) u S in the matrix units, S
the sum of the absolute products; bias, activation (slope at most 1.13, 4e-6 of
z relative and u |z| absolute at most, z within 12) and residual add a few u;
an output in BF16 is rounded by 2^-8 relative; the gradients behind an
activation take dz in BF16, which adds 2^-8 of their S.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=g.device) * scale).to(BF16)


def _wide(t, extra):
    """t as the left part of rows `extra` wider, the rest NaN."""
    w = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def _product(a, b):
    """a b^T and the same of absolute values, in float64."""
    a, b = a.double(), b.double()
    return a @ b.T.contiguous(), a.abs() @ b.abs().T.contiguous()


def _close(got, want, err, what):
    if got.dtype == BF16:
        err = err + 2.0 ** -8 * (want.abs() + err)
    bad = ~((got.double() - want).abs() <= err + 1e-38)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def _choice(product, m, n, k, groups=1):
    c = _fg8().bf16_tile_choice(product, m, n, k, groups)
    return c["bm"], c["bn"], c["splits"] > 1


def _act(name, z):
    """(act(z), act'(z))"""
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p + z * p * (1 - p)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


FEW, THIN, FLAT, LOW, HIGH, MID, BIG = (16, 16), (16, 64), (32, 64), (64, 64), (128, 64), (128, 128), (256, 256)
DUO = (128, 256)

FORWARD = [
    (FEW, False, 3, 200, 1032), (FEW, False, 8, 37, 4096),
    (THIN, False, 16, 12803, 264), (THIN, True, 11, 70, 4168), (THIN, True, 16, 64, 4160),
    (FLAT, False, 29, 12801, 72), (FLAT, True, 17, 200, 1000), (FLAT, True, 32, 515, 2048),
    (LOW, False, 130, 3001, 72), (LOW, True, 200, 264, 2048),
    (HIGH, False, 300, 515, 136), (HIGH, True, 290, 128, 2056),
    (MID, False, 1024, 7168, 136), (MID, False, 1030, 7163, 136), (MID, False, 2040, 4096, 200),
    (BIG, False, 2100, 8000, 72), (BIG, False, 1281, 7161, 200)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("tile,split,m,n,k", FORWARD)
def test_dense_forward(dev, tile, split, m, n, k, act):
    print(f"dense forward {m}x{n}x{k} {act}, tile {tile}", flush=True)
    assert _choice("gemm_bf16_epilogue", m, n, k) == (*tile, split)
    g = torch.Generator(device=dev).manual_seed(m + 7 * n)
    x, w = _bf16(g, m, k), _bf16(g, n, k, scale=k ** -0.5)
    bias, res = torch.randn(n, generator=g, device=dev), _bf16(g, m, n)
    z0, s = _product(x, w)
    fg8 = _fg8()
    if act == "none":                       # nothing but the product
        e = 2 * (k + 1) * U * s
        for out in (BF16, F32):
            _close(fg8.gemm_bf16_epilogue(_wide(x, 8), w, out_dtype=out), z0, e, f"x w^T in {out}")
    z0, s = z0 + bias.double(), s + bias.double().abs()
    e = 2 * (k + 1) * U * s + 2 * U * z0.abs()
    a, _ = _act(act, z0)
    e_a = 1.13 * e + 4e-6 * a.abs() + 2 * U * z0.abs()
    y, z = fg8.gemm_bf16_epilogue(_wide(x, 8), w, bias, _wide(res, 3 if n % 2 else 8), activation=act, save_z=True)
    _close(z, z0, e, "z")
    want = a + res.double()
    _close(y, want, e_a + 2 * U * (want.abs() + res.double().abs()), "y")
    wide = torch.full((m, n + 5), 7.0, dtype=F32, device=dev)
    fg8.gemm_bf16_epilogue(x, w, bias, activation=act, out=wide[:, :n])
    _close(wide[:, :n], a, e_a, "FP32 y in wider rows")
    assert bool((wide[:, n:] == 7).all()), "columns past n were written"


# the tiles of dx [m][k], summed over n, and of dw [n][k], summed over m
BACKWARD = [
    (THIN, True, MID, False, 5, 1000, 264), (FLAT, True, MID, False, 17, 1000, 200), (FLAT, False, MID, False, 32, 72, 12808),
    (LOW, True, MID, False, 64, 1040, 520), (HIGH, False, MID, False, 400, 200, 520),
    (MID, False, MID, True, 1024, 136, 7168), (BIG, False, MID, True, 2100, 72, 8000),
    (HIGH, True, BIG, False, 300, 4096, 2056), (HIGH, True, BIG, False, 300, 4099, 2056),
    (HIGH, False, MID, True, 2000, 200, 264), (LOW, True, MID, False, 200, 2048, 512), (BIG, False, BIG, False, 2300, 4104, 4104)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dx_tile,dx_split,dw_tile,dw_split,m,n,k", BACKWARD)
def test_dense_backward(dev, dx_tile, dx_split, dw_tile, dw_split, m, n, k, act):
    print(f"dense backward {m}x{n}x{k} {act}, tiles {dx_tile} {dw_tile}", flush=True)
    assert _choice("dx", m, n, k) == (*dx_tile, dx_split) and _choice("dw", m, n, k) == (*dw_tile, dw_split)
    g = torch.Generator(device=dev).manual_seed(m + 7 * n + k)
    x, w, dy = _bf16(g, m, k), _bf16(g, n, k), _bf16(g, m, n)
    z = _bf16(g, m, n, scale=2.0)
    dz = dy.double() * _act(act, z.double())[1]
    # dz before its rounding: the slope's terms are below |z| + 2
    term = dy.double().abs() * (z.double().abs() + 2) * (4e-6 if act != "none" else 0.0)
    off = term + (2.0 ** -8 * (dz.abs() + term) if act != "none" else 0.0)
    size = dz.abs() + off
    dx, dw, db = _fg8().gemm_bf16_epilogue_backward(_wide(dy, 3 if n % 2 else 8), _wide(x, 16), w, z, activation=act, dw_dtype=F32)
    W, X = w.double().abs(), x.double().abs()
    _close(dx, dz @ w.double(), off @ W + 2 * (n + 1) * U * (size @ W), "dx")
    t = lambda v: v.T.contiguous()   # noqa: E731
    _close(dw, t(dz) @ x.double(), t(off) @ X + 2 * (m + 1) * U * (t(size) @ X), "dw")
    _close(db, dz.sum(0), term.sum(0) + (m + 1) * U * (dz.abs() + term).sum(0), "dbias")


# experts, rows on average, n, k; the tile of the forward pass, then of the input gradient
GROUPED = [
    (FEW, THIN, 6, 5, 200, 1032), (THIN, THIN, 9, 7, 520, 4104), (FLAT, FLAT, 5, 20, 200, 264), (LOW, LOW, 7, 60, 264, 520),
    (HIGH, HIGH, 4, 300, 1000, 1016), (MID, MID, 16, 120, 2056, 2048), (BIG, BIG, 4, 750, 3000, 2816)]


@pytest.mark.parametrize("forward,dgrad,experts,per,n,k", GROUPED)
def test_grouped(dev, forward, dgrad, experts, per, n, k):
    rows = experts * per
    print(f"grouped {experts} runs of {per} rows, {n}x{k}, tiles {forward} {dgrad}", flush=True)
    assert _choice("grouped_gemm_bf16", rows, n, k, experts)[:2] == forward
    assert _choice("grouped_gemm_bf16_dgrad", rows, n, k, experts)[:2] == dgrad
    g = torch.Generator(device=dev).manual_seed(rows + n)
    cut = torch.sort(torch.randint(0, rows + 1, (experts + 1,), generator=g, device=dev)).values    # rows of no run at both ends
    off = cut.tolist()
    x, dy, w = _bf16(g, rows, k), _bf16(g, rows, n), _bf16(g, experts, n, k)
    o = cut.to(torch.int32)
    fg8 = _fg8()
    for out in (BF16, F32):
        y = fg8.grouped_gemm_bf16(_wide(x, 8), w, o, out_dtype=out)
        dx = fg8.grouped_gemm_bf16_dgrad(_wide(dy, 16), w, o, out_dtype=out)
        for e in range(experts):
            a, b = off[e], off[e + 1]
            want, s = _product(x[a:b], w[e])
            _close(y[a:b], want, 2 * (k + 1) * U * s, f"y of expert {e}")
            want, s = _product(dy[a:b], w[e].T)
            _close(dx[a:b], want, 2 * (n + 1) * U * s, f"dx of expert {e}")
        for t in (y, dx):
            assert not t[:off[0]].any() and not t[off[-1]:].any(), "rows of no run"


@pytest.mark.parametrize("tile,experts,per,n,k", [(MID, 5, 140, 520, 264), (MID, 4, 1024, 1040, 1032), (DUO, 40, 22, 1800, 1544),
                                                  (BIG, 2, 2100, 4096, 4104)])
def test_grouped_wgrad(dev, tile, experts, per, n, k):
    rows = experts * per
    print(f"grouped wgrad {experts} runs of {per} rows, {n}x{k}, tile {tile}", flush=True)
    assert _choice("grouped_gemm_bf16_wgrad", rows, n, k, experts)[:2] == tile
    g = torch.Generator(device=dev).manual_seed(rows + n)
    cut = torch.sort(torch.randint(0, rows + 1, (experts + 1,), generator=g, device=dev)).values
    off = cut.tolist()
    x, dy = _bf16(g, rows, k), _bf16(g, rows, n)
    want = []
    for a, b in zip(off, off[1:]):
        want.append((_product(dy[a:b].T, x[a:b].T), b - a))
    for t in (x, dy):                       # what rows of no run hold is not read
        t[:off[0]] = float("nan")
        t[off[-1]:] = float("inf")
    for out in (BF16, F32):
        dw = _fg8().grouped_gemm_bf16_wgrad(_wide(dy, 8), _wide(x, 8), cut.to(torch.int32), out_dtype=out)
        for e, ((exact, s), length) in enumerate(want):
            _close(dw[e], exact, 2 * (length + 1) * U * s, f"dw of expert {e}")
