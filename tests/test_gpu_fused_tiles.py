"""Every tile of the gated products and of the loss's logits at a size that is
given it, the choice asserted: a changed rule cannot leave an instance of the
kernels untested.

References are float64 products on the GPU.  Bounds, with u = 2^-24: a sum of K
products of BF16 values is off by at most e = 2 (K + 1) u S, S the sum of the
absolute products.  h = act(g) up: 1.13 e_g (|up| + e_up) + |act(g)| e_up, and 2^-19 of
its value for the activation's own arithmetic (absolute below 2^-19).  lse: no more
than its largest logit's error, 2^-17 for the exponentials, (V + 8) u for their sum
and 2 u |lse|; the loss besides by its target's e and 4 u of both.  A probability is
off by a factor of e^(e + 2^-17), dl so by (e + 2^-17)(p + 2^-22) |dloss| + 2^-22 |dl|,
and by 2^-8 of itself where it is rounded to BF16 (2^-15 in two parts).  An output in
BF16 is rounded by 2^-8 relative.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
FEW, FLAT, LOW, HIGH, MID, BIG = (16, 32), (32, 64), (64, 64), (128, 64), (128, 128), (256, 256)
SLAB = (64, 128)


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
    """a b^T and the bound of its error, in float64."""
    a, b = a.double(), b.double().T.contiguous()
    return a @ b, 2 * (a.shape[1] + 1) * U * (a.abs() @ b.abs())


def _close(got, want, err, what):
    if got.dtype == BF16:
        err = err + 2.0 ** -8 * (want.abs() + err)
    bad = ~((got.double() - want).abs() <= err + 1e-38)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def _choice(product, m, n, k, groups=1):
    c = _fg8().bf16_tile_choice(product, m, n, k, groups)
    return (c["bm"], c["bn"]), c["splits"] > 1


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z.clamp(min=0) if name == "relu" else z


def _gated(act, z, e):
    n = z.shape[1] // 2
    a, up, eg, eu = _act(act, z[:, :n]), z[:, n:], e[:, :n], e[:, n:]
    return a * up, 1.13 * eg * (up.abs() + eu) + a.abs() * eu + 2.0 ** -19 * (a.abs() + 2.0 ** -19) * up.abs()


GATED = [(FEW, False, 3, 43, 520), (FEW, False, 8, 500, 4096), (FLAT, True, 20, 72, 2056), (FLAT, False, 31, 77, 200), (LOW, True, 100, 133, 1000),
         (HIGH, False, 300, 264, 328), (MID, False, 300, 8200, 72), (MID, False, 515, 5003, 136), (MID, False, 384, 8192, 64),
         (BIG, False, 300, 12001, 72), (BIG, False, 1500, 5000, 200), (BIG, False, 2101, 5003, 72)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tile,split,m,n,k", GATED)
def test_gated(dev, tile, split, m, n, k, act):
    print(f"gated {m}x{n}x{k} {act}, tile {tile}", flush=True)
    assert _choice("gemm_bf16_gated", m, n, k) == (tile, split)
    fg8, g = _fg8(), torch.Generator(device=dev).manual_seed(m + 7 * n)
    x, w = _bf16(g, m, k), _bf16(g, 2 * n, k, scale=k ** -0.5)
    z0, e = _product(x, w)
    want, err = _gated(act, z0, e)
    h, z = fg8.gemm_bf16_gated(_wide(x, 8), w, activation=act, save_z=True)
    _close(h, want, err, "h")
    _close(z, z0, e, "z")
    assert torch.equal(fg8.gemm_bf16_gated(x, w, activation=act), h)
    wide = torch.full((m, n + 5), 7.0, dtype=F32, device=dev)
    fg8.gemm_bf16_gated(x, w, activation=act, out=wide[:, :n])
    _close(wide[:, :n], want, err, "FP32 h in wider rows")
    assert bool((wide[:, n:] == 7).all()), "columns past n were written"


# rows before the first run and after the last one, runs' lengths, n, k
RUNS = [(FEW, 1, 2, [0, 9, 3, 1, 0, 12], 43, 520), (FLAT, 0, 3, [17, 0, 40, 33], 77, 4168), (LOW, 2, 0, [70, 1, 100], 72, 136),
        (HIGH, 0, 1, [300, 513, 2], 77, 136), (MID, 3, 5, [(37 * e * e) % 83 for e in range(32)], 523, 136),
        (MID, 0, 0, [128] * 16, 1024, 64), (BIG, 3, 2, [700, 0, 255, 257, 1, 300, 390, 600], 921, 72),
        (BIG, 1, 0, [900, 513, 0, 1023, 256, 700, 1, 600], 2203, 72)]


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("tile,before,after,counts,n,k", RUNS)
def test_gated_runs(dev, tile, before, after, counts, n, k, act):
    rows = before + sum(counts) + after
    print(f"gated runs {counts} {n}x{k} {act}, tile {tile}", flush=True)
    assert _choice("grouped_gemm_bf16_gated", rows, n, k, len(counts)) == (tile, False)
    fg8, g = _fg8(), torch.Generator(device=dev).manual_seed(rows + 7 * n)
    x, w = _bf16(g, rows, k), _bf16(g, len(counts), 2 * n, k, scale=k ** -0.5)
    z0, e = torch.zeros(rows, 2 * n, dtype=F64, device=dev), torch.zeros(rows, 2 * n, dtype=F64, device=dev)
    off = [before]
    for i, c in enumerate(counts):
        a, b = off[-1], off[-1] + c
        z0[a:b], e[a:b] = _product(x[a:b], w[i])
        off.append(b)
    x[:before] = x[off[-1]:] = float("nan")
    want, err = _gated(act, z0, e)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev)
    for out in (BF16, F32):
        h, z = fg8.grouped_gemm_bf16_gated(_wide(x, 8), w, offsets, activation=act, save_z=True, out_dtype=out)
        _close(h, want, err, "h")
        _close(z, z0, e, "z")
        for t in (h, z):
            assert not t[:before].any() and not t[off[-1]:].any(), "rows of no run"


# 128 x 128 tiles up to one a CU (three stages) and beyond (two); big ones, more than
# one a CU in the last
LOSS = [(SLAB, False, 61, 901, 136), (SLAB, True, 53, 300, 2048), (MID, False, 130, 1001, 328), (MID, True, 200, 2000, 2120),
        (MID, False, 130, 16601, 72), (MID, False, 257, 11000, 200), (MID, False, 512, 12800, 64), (BIG, False, 700, 16601, 72),
        (BIG, False, 1100, 8200, 264), (BIG, False, 1101, 20003, 72)]


@pytest.mark.parametrize("tile,split,m,v,k", LOSS)
def test_loss(dev, tile, split, m, v, k):
    print(f"loss {m}x{v}x{k}, tile {tile}", flush=True)
    for product in ("linear_cross_entropy", "linear_cross_entropy_backward"):
        assert _choice(product, m, v, k) == (tile, split)
    fg8, g = _fg8(), torch.Generator(device=dev).manual_seed(m + 7 * v)
    x, w = _bf16(g, m, k), _bf16(g, v, k, scale=3 * k ** -0.5)
    t = torch.randint(0, v, (m,), device=dev, generator=g)
    t[::5], t[3], t[6] = -100, v, v - 1
    live = (t >= 0) & (t < v)
    at, rows = t.clamp(0, v - 1), torch.arange(m, device=dev)
    l, e = _product(x, w)
    lse0 = torch.logsumexp(l, 1)
    E = e.amax(1) + 2.0 ** -17 + (v + 8) * U + 2 * U * lse0.abs()
    loss, lse = fg8.linear_cross_entropy(_wide(x, 8), w, t)
    _close(lse, lse0, E, "lse")
    _close(loss, (lse0 - l[rows, at]) * live, (E + e[rows, at] + 4 * U * (lse0.abs() + l[rows, at].abs())) * live, "loss")

    dloss = 0.5 + torch.rand(m, device=dev, generator=g)
    clean = torch.where(live, dloss, 0.0).double()[:, None]
    p = torch.exp(l - lse.double()[:, None]) * live[:, None]
    dl = p.clone()
    dl[rows, at] -= 1.0
    dl *= clean
    ed = (e + 2.0 ** -17) * (p + 2.0 ** -22) * clean + 2.0 ** -22 * dl.abs()
    xd, wd = x.double(), w.double()
    dloss[~live] = float("nan")
    for dtype, step in ((BF16, 2.0 ** -8), (F32, 2.0 ** -15)):
        dx, dw = fg8.linear_cross_entropy_backward(dloss, _wide(x, 8), w, t, lse, dw_dtype=dtype)
        r = ed + 2.0 ** -8 * (dl.abs() + ed)
        _close(dx, dl @ wd, r @ wd.abs() + 2 * (v + 1) * U * ((dl.abs() + r) @ wd.abs()), f"dx beside dw in {dtype}")
        r, parts = ed + step * (dl.abs() + ed), 1 if dtype == BF16 else 2
        r, size = r.T.contiguous() @ xd.abs(), (dl.abs() + r).T.contiguous() @ xd.abs()
        _close(dw, dl.T.contiguous() @ xd, r + parts * 2 * (m + 1) * U * size, f"dw in {dtype}")


def test_both_tiles_of_128_rows_are_above(dev):
    """(which of the two it is follows from the tiles a CU has)"""
    cus = torch.cuda.get_device_properties(dev).multi_processor_count
    tiles = [-(-m // 128) * -(-v // 128) for tile, _, m, v, _ in LOSS if tile == MID]
    assert min(tiles) <= cus < max(tiles) <= 2 * cus and sum(t > cus for t in tiles) >= 2
