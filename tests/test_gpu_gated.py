"""The gated BF16 products, dense and over ragged runs, forward and backward,
against the float64 forms.

Bounds.  Each sum of K products of BF16 values is off by e = 2 (K + 1) 2^-24 S
at most (S the sum of the absolute products; any order of the additions, and
the matrix unit may cut where FP32 rounds).  The activations' slopes lie below
1.13 and act(z) within (1, 1 + |z|) |z|; hence h = act(g) u is off by
1.13 e_g (|u| + e_u) + |act(g)| e_u, and 2^-19 of its value for the activation's
own arithmetic.  A BF16 output adds 2^-8 of the value, half a step.
Backward, dz is computed from the saved z in FP32 (2^-18 of the values involved,
(|z_up| 1.13 + |act|) |dh|), rounded to BF16 by up to 2^-8 relative, or to 2^-15 in
two parts for a float32 dw; the products' terms are off by as much.
"""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 6133 * k for i, k in enumerate(key)) + 11)


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(BF16)


def _np(t):
    return t.detach().cpu().double().numpy()


def _strided(t, dev, extra):
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=dev)
    wide[:, :t.shape[1]] = t.to(dev)
    return wide[:, :t.shape[1]]


def _sum_error(k, s):
    return 2 * (k + 1) * 2.0 ** -24 * s


def _check(got, want, err, what):
    g = _np(got)
    rounding = 2.0 ** -8 * (np.abs(want) + err) if got.dtype == BF16 else 0.0
    bad = ~(np.abs(g - want) <= err + rounding + 1e-38)
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} for {want[bad][0]}")


def _h_error(act, z, ez):
    n = z.shape[1] // 2
    g, u, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
    a = np.abs(layer.activation(act, g))
    return 1.13 * eg * (np.abs(u) + eu) + a * eu + 2.0 ** -19 * (a + 2.0 ** -19) * np.abs(u)


# m, n, k: odd widths, one row, splits of k, every tile
DENSE = [(1, 16, 8), (1, 37, 520), (1, 1000, 2048), (3, 129, 72), (17, 64, 328), (33, 136, 4096), (64, 256, 7168), (70, 4, 64),
         (130, 200, 264), (257, 133, 136), (300, 1060, 200), (1200, 2050, 136), (2049, 2056, 72)]


@pytest.mark.parametrize("case", range(len(DENSE)))
def test_dense_forward(dev, case):
    m, n, k = DENSE[case]
    act = ["silu", "gelu", "relu", "none"][case % 4]
    out = [BF16, F32][case // 4 % 2]
    print(f"gated {m}x{n}x{k} {act} {out}", flush=True)
    g = _gen(1, case)
    x, w = _bf16(g, m, k), _bf16(g, 2 * n, k, scale=k ** -0.5)
    z, s = layer.dense(_np(x), _np(w))
    ez = _sum_error(k, s)
    want = layer.gated(act, z)
    wide = torch.full((m, n + 3), 7.0, dtype=out, device=dev)
    h = wide[:, :n] if case % 3 == 1 and m > 1 else None
    got, gz = _fg8().gemm_bf16_gated(_strided(x, dev, 8 * (case % 2)), w.to(dev), activation=act, save_z=True, out_dtype=out, out=h)
    _check(gz, z, ez, "z")
    _check(got, want, _h_error(act, z, ez), "h")
    if h is not None:
        assert (wide[:, n:] == 7).all(), "columns past n were written"
    again = _fg8().gemm_bf16_gated(_strided(x, dev, 0), w.to(dev), activation=act, out_dtype=out)
    assert torch.equal(again, got), "without z the same bits"


# counts, rows before the first run, rows after the last, n, k
RUNS = [
    ([1], 0, 0, 8, 8),
    ([0, 0, 5], 0, 0, 37, 64),
    ([3, 0, 17, 1], 2, 3, 72, 136),
    ([16, 16], 0, 0, 200, 2048),
    ([64, 1, 65, 0, 63], 1, 0, 104, 200),
    ([130, 257, 0, 1, 300], 0, 70, 129, 328),
    ([0] * 70 + [9] + [0] * 60 + [33], 0, 4, 40, 96),
    ([1030, 0, 900, 1111, 1055], 3, 5, 2052, 72),
]


def _offsets(counts, before):
    return np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)


@pytest.mark.parametrize("case", range(len(RUNS)))
def test_runs_forward(dev, case):
    counts, before, after, n, k = RUNS[case]
    off = _offsets(counts, before)
    rows, act, out = int(off[-1]) + after, ["silu", "relu", "gelu"][case % 3], [BF16, F32][case % 2]
    print(f"gated runs case {case} rows {rows} n {n} k {k} {act} {out}", flush=True)
    g = _gen(2, case)
    x, w = _bf16(g, rows, k), _bf16(g, len(counts), 2 * n, k, scale=k ** -0.5)
    z, s = layer.grouped(_np(x), _np(w), off)
    ez = _sum_error(k, s)
    x = _strided(x, dev, 8 * (case % 3))
    x[:before] = float("nan")              # rows of no run are not read
    x[int(off[-1]):] = float("nan")
    h, gz = _fg8().grouped_gemm_bf16_gated(x, w.to(dev), torch.from_numpy(off).to(dev), activation=act, save_z=True, out_dtype=out)
    z[:before] = z[off[-1]:] = 0
    _check(gz, z, ez, "z")
    _check(h, layer.gated(act, z), _h_error(act, z, ez), "h")


def _dz(act, dh, z):
    """dz and how far the kernel's FP32 dz may be from it."""
    n = z.shape[1] // 2
    dz = layer.gated_dz(act, dh, z)
    a, u = np.abs(layer.activation(act, z[:, :n])), np.abs(z[:, n:])
    return dz, 2.0 ** -18 * np.concatenate([np.abs(dh) * u * 1.13, np.abs(dh) * a], 1)


@pytest.mark.parametrize("dw_dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(DENSE)))
def test_dense_backward(dev, case, dw_dtype):
    m, n, k = DENSE[case]
    act = ["gelu", "silu", "none", "relu"][case % 4]
    print(f"gated backward {m}x{n}x{k} {act} {dw_dtype}", flush=True)
    g = _gen(3, case)
    x, w, dh, z = _bf16(g, m, k), _bf16(g, 2 * n, k, scale=k ** -0.5), _bf16(g, m, n), _bf16(g, m, 2 * n, scale=1.5)
    dz, ed = _dz(act, _np(dh), _np(z))
    ed8, ed15 = ed + 2.0 ** -8 * (np.abs(dz) + ed), ed + 2.0 ** -15 * (np.abs(dz) + ed)
    ax, aw = np.abs(_np(x)), np.abs(_np(w))
    dx, dw = _fg8().gemm_bf16_gated_backward(_strided(dh, dev, case % 3), _strided(x, dev, 8 * (case % 2)), w.to(dev),
                                             z.to(dev), activation=act, dw_dtype=dw_dtype)
    size = np.abs(dz) + ed8
    _check(dx, dz @ _np(w), ed8 @ aw + _sum_error(2 * n, size @ aw), "dx")
    e = (ed8 if dw_dtype == BF16 else ed15).T @ ax + (1 if dw_dtype == BF16 else 2) * _sum_error(m, size.T @ ax)
    _check(dw, dz.T @ _np(x), e, "dw")
    only = _fg8().gemm_bf16_gated_backward(dh.to(dev), x.to(dev), w.to(dev), z.to(dev), activation=act, dw_dtype=dw_dtype,
                                           needs=(False, True))
    assert only[0] is None and torch.equal(only[1], dw)


@pytest.mark.parametrize("dw_dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_runs_backward(dev, case, dw_dtype):
    counts, before, after, n, k = RUNS[case]
    off = _offsets(counts, before)
    rows, act = int(off[-1]) + after, ["silu", "gelu", "relu"][case % 3]
    print(f"gated backward runs case {case} rows {rows} n {n} k {k} {act} {dw_dtype}", flush=True)
    g = _gen(4, case)
    x, w = _bf16(g, rows, k), _bf16(g, len(counts), 2 * n, k, scale=k ** -0.5)
    dh, z = _bf16(g, rows, n), _bf16(g, rows, 2 * n, scale=1.5)
    dz, ed = _dz(act, _np(dh), _np(z))
    ed8, ed15 = ed + 2.0 ** -8 * (np.abs(dz) + ed), ed + 2.0 ** -15 * (np.abs(dz) + ed)
    size, aw, ax = np.abs(dz) + ed8, np.abs(_np(w)), np.abs(_np(x))
    x, dh, z = x.to(dev), dh.to(dev), z.to(dev)
    x[:before] = dh[:before] = z[:before] = float("nan")
    x[int(off[-1]):] = dh[int(off[-1]):] = z[int(off[-1]):] = float("nan")
    dx, dw = _fg8().grouped_gemm_bf16_gated_backward(dh, x, w.to(dev), z, torch.from_numpy(off).to(dev), activation=act,
                                                     dw_dtype=dw_dtype)
    want, _ = layer.grouped_dgrad(dz, _np(w), off)
    _check(dx, want, layer.grouped_dgrad(ed8, aw, off)[0] + _sum_error(2 * n, layer.grouped_dgrad(size, aw, off)[0]), "dx")
    xs = np.where(np.isnan(_np(x)), 0, _np(x))
    want, _ = layer.grouped_wgrad(dz, xs, off)
    e = layer.grouped_wgrad(ed8 if dw_dtype == BF16 else ed15, ax, off)[0]
    e = e + (1 if dw_dtype == BF16 else 2) * _sum_error(max(counts), layer.grouped_wgrad(size, ax, off)[0])
    _check(dw, want, e, "dw")


def test_gradient_by_differences(dev):
    """d(sum of dh h) along a direction by central differences of the forward
    pass in FP32 out, against dx and dw: a step of 2^-4 leaves an error of the
    third derivative's size, some 2^-8 of the value, and the BF16 roundings of
    dx and dw as much again: 0.02 of the gradient's length times the direction's."""
    m, n, k = 24, 40, 64
    g = _gen(5)
    x, w = _bf16(g, m, k), _bf16(g, 2 * n, k, scale=k ** -0.5)
    dh = _bf16(g, m, n)
    fg8 = _fg8()
    _, z = fg8.gemm_bf16_gated(x.to(dev), w.to(dev), save_z=True)
    dx, dw = fg8.gemm_bf16_gated_backward(dh.to(dev), x.to(dev), w.to(dev), z)

    def value(xs, ws):
        h = fg8.gemm_bf16_gated(xs.to(dev), ws.to(dev), out_dtype=F32)
        return float((h.cpu().double() * dh.double()).sum())
    for t, grad, other in ((x, dx, "x"), (w, dw, "w")):
        d = _bf16(g, *t.shape, scale=float(t.float().std()))
        lo, hi = (t.float() - d.float() / 16).to(BF16), (t.float() + d.float() / 16).to(BF16)
        step = (hi.double() - lo.double())
        diff = value(hi, w) - value(lo, w) if other == "x" else value(x, hi) - value(x, lo)
        along = float((grad.cpu().double() * step).sum())
        assert abs(diff - along) <= 0.02 * float(grad.cpu().double().norm() * step.norm()), (other, diff, along)


def test_empty(dev):
    fg8 = _fg8()
    x, w = torch.empty(0, 64, dtype=BF16, device=dev), torch.ones(32, 64, dtype=BF16, device=dev)
    h, z = fg8.gemm_bf16_gated(x, w, save_z=True)
    assert h.shape == (0, 16) and z.shape == (0, 32)
    dx, dw = fg8.gemm_bf16_gated_backward(h, x, w, z)
    assert dx.shape == (0, 64) and not dw.any()
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    w = torch.ones(2, 32, 64, dtype=BF16, device=dev)
    h, z = fg8.grouped_gemm_bf16_gated(x, w, off, save_z=True)
    dx, dw = fg8.grouped_gemm_bf16_gated_backward(h, x, w, z, off)
    assert h.shape == (0, 16) and dw.shape == w.shape and not dw.any()


def test_captured(dev):
    """Forward and backward in one graph, split products among them, replayed
    with eager calls between."""
    fg8 = _fg8()
    g = _gen(6)
    x, w, dh = _bf16(g, 40, 4096).to(dev), _bf16(g, 264, 4096, scale=4096 ** -0.5).to(dev), _bf16(g, 40, 132).to(dev)

    def both():
        h, z = fg8.gemm_bf16_gated(x, w, save_z=True)
        return (h, *fg8.gemm_bf16_gated_backward(dh, x, w, z, dw_dtype=F32))
    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert all(torch.equal(a, b) for a, b in zip(both(), want))


@pytest.mark.parametrize("experts,rows,n,k,tile", [(64, 1300, 1024, 1024, (128, 256)), (4, 8420, 2048, 2048, (256, 256))])
def test_float_weight_gradient_of_many_tiles(dev, experts, rows, n, k, tile):
    """A float32 dw of row runs where both of its products take the larger tiles,
    against float32 products of the same dz on the GPU (TF32 is off): its dz is
    2^-15 off, its sums and theirs 4 (rows + 1) 2^-24 of the absolute sums."""
    fg8 = _fg8()
    choice = fg8.bf16_tile_choice("grouped_gemm_bf16_wgrad", rows, 2 * n, k, groups=experts)
    assert (choice["bm"], choice["bn"]) == tile
    g = torch.Generator(device=dev).manual_seed(experts)
    x, dh, z = (torch.randn(rows, c, device=dev, generator=g).to(BF16) for c in (k, n, 2 * n))
    w = torch.zeros(experts, 2 * n, k, dtype=BF16, device=dev)
    cuts = torch.sort(torch.randperm(rows, generator=torch.Generator().manual_seed(1))[:experts - 1]).values
    off = torch.cat([torch.tensor([0]), cuts, torch.tensor([rows])]).to(torch.int32)
    _, dw = fg8.grouped_gemm_bf16_gated_backward(dh, x, w, z, off.to(dev), needs=(False, True))
    zg, zu = z[:, :n].double(), z[:, n:].double()
    p = torch.sigmoid(zg)
    dz = torch.cat([dh.double() * zu * (p + zg * p * (1 - p)), dh.double() * zg * p], 1).float()
    size = torch.cat([dh.float().abs() * zu.float().abs() * 1.13, dh.float().abs() * (zg * p).float().abs()], 1)
    for e in (0, 1, experts // 2, experts - 1):
        r = slice(int(off[e]), int(off[e + 1]))
        want, most = dz[r].T @ x[r].float(), size[r].T @ x[r].float().abs()
        assert ((dw[e] - want).abs() <= (2.0 ** -15 + 2.0 ** -17 + 4 * (r.stop - r.start + 1) * 2.0 ** -24) * most + 1e-30).all(), e
