"""The BF16 products (ragged expert products and the dense product with an
epilogue, forward and backward) against the float64 forms.

Bounds.  An FP32 sum of K products of BF16 values (exact in FP32) is off by at
most (K + 1) 2^-24 S in any order of the additions, S the sum of the absolute
products; the matrix unit may truncate where FP32 rounds, hence twice that:
e = 2 (K + 1) 2^-24 S.  A bias, residual or activation adds a few roundings of
2^-24 relative, and the activations' hardware exp and erff some ulp more:
2^-20 of the values involved.  Each of the four activations has a slope below
1.13.  A BF16 output is then rounded by at most 2^-8 relative (half an ulp, 2^(e-8),
of a value of 2^e or more).  The backward products take dz rounded to BF16, so
each of their terms may be off by 2^-8: 2^-8 S more.
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
    return torch.Generator().manual_seed(sum((i + 1) * 7919 * k for i, k in enumerate(key)) + 5)


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(BF16)


def _np(t):
    return t.detach().cpu().double().numpy()


def _strided(t, dev, extra, poison=float("nan")):
    """t on the device as the left part of rows `extra` elements wider, whose
    other part holds `poison`."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), poison, dtype=t.dtype, device=dev)
    wide[:, :t.shape[1]] = t.to(dev)
    return wide[:, :t.shape[1]]


def _sum_error(k, s):
    return 2 * (k + 1) * 2.0 ** -24 * s


def _check(got, want, err, what):
    rounding = 2.0 ** -8 * (np.abs(want) + err) if got.dtype == BF16 else 0.0
    g = _np(got)
    bad = ~(np.abs(g - want) <= err + rounding + 1e-38)
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} off, first at "
                           f"{np.argwhere(bad)[0]}: {g[bad][0]} for {want[bad][0]}")


def _offsets(counts, before=0):
    return np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)


# counts, rows before the first run, rows after the last, n, k
RUNS = [
    ([1], 0, 0, 8, 8),
    ([0, 0, 5], 0, 0, 40, 64),
    ([3, 0, 17, 1], 2, 3, 136, 72),                    # rows of no run on both sides
    ([16, 16], 0, 0, 64, 128),
    ([64, 1, 65, 0, 63], 1, 0, 200, 200),
    ([130, 257, 0, 1, 300], 0, 70, 264, 328),
    ([0] * 70 + [9] + [0] * 60 + [33], 0, 4, 72, 96),  # more experts than a wave has lanes
    ([1030, 0, 900, 1111, 1055], 3, 5, 4096, 136),     # the largest tiles
]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_grouped_forward(dev, case, out):
    counts, before, after, n, k = RUNS[case]
    off = _offsets(counts, before)
    rows = int(off[-1]) + after
    print(f"grouped forward case {case} rows {rows} n {n} k {k} out {out}", flush=True)
    g = _gen(1, case)
    x, w = _bf16(g, rows, k), _bf16(g, len(counts), n, k)
    want, s = layer.grouped(_np(x), _np(w), off)
    y = _fg8().grouped_gemm_bf16(_strided(x, dev, 8 * (case % 3)), w.to(dev), torch.from_numpy(off).to(dev), out_dtype=out)
    _check(y, want, _sum_error(k, s), "y")


@pytest.mark.parametrize("n", [1, 3, 37, 129])
def test_grouped_forward_odd_columns(dev, n):
    off = _offsets([5, 40, 0, 20], 1)
    g = _gen(2, n)
    x, w = _bf16(g, 70, 88), _bf16(g, 4, n, 88)
    want, s = layer.grouped(_np(x), _np(w), off)
    wide = torch.full((70, n + 5), 7.0, dtype=BF16, device=dev)
    _fg8().grouped_gemm_bf16(x.to(dev), w.to(dev), torch.from_numpy(off).to(dev), out=wide[:, :n])
    _check(wide[:, :n], want, _sum_error(88, s), "y")
    assert (wide[:, n:] == 7).all(), "columns past n were written"


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_grouped_dgrad(dev, case, out):
    counts, before, after, n, k = RUNS[case]
    if case == len(RUNS) - 1:
        n, k = k, n                                    # many columns of dx: the largest tiles
    off = _offsets(counts, before)
    rows = int(off[-1]) + after
    print(f"grouped dgrad case {case} rows {rows} n {n} k {k} out {out}", flush=True)
    g = _gen(3, case)
    dy, w = _bf16(g, rows, n), _bf16(g, len(counts), n, k)
    want, s = layer.grouped_dgrad(_np(dy), _np(w), off)
    dx = _fg8().grouped_gemm_bf16_dgrad(_strided(dy, dev, 8 * (case % 2)), w.to(dev), torch.from_numpy(off).to(dev), out_dtype=out)
    _check(dx, want, _sum_error(n, s), "dx")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_grouped_wgrad(dev, case, out):
    counts, before, after, n, k = RUNS[case]
    if case == len(RUNS) - 1:
        n, k = 2040, 2048
    off = _offsets(counts, before)
    rows = int(off[-1]) + after
    print(f"grouped wgrad case {case} rows {rows} n {n} k {k} out {out}", flush=True)
    g = _gen(4, case)
    dy, x = _bf16(g, rows, n), _bf16(g, rows, k)
    want, s = layer.grouped_wgrad(_np(dy), _np(x), off)
    # what rows of no run hold takes no part in any sum
    for t in (dy, x):
        t[:before] = float("nan")
        t[rows - after:] = float("inf")
    dw = _fg8().grouped_gemm_bf16_wgrad(_strided(dy, dev, 8), _strided(x, dev, 16), torch.from_numpy(off).to(dev), out_dtype=out)
    longest = max(counts)
    _check(dw, want, _sum_error(longest, s), "dw")


def test_grouped_one_experts_nan_stays_with_it(dev):
    """NaN and infinite rows of one expert reach no other expert's outputs."""
    off = _offsets([70, 3, 61])
    g = _gen(5)
    x, dy, w = _bf16(g, 134, 72), _bf16(g, 134, 80), _bf16(g, 3, 80, 72)
    x[70:73], dy[70:73] = float("nan"), float("inf")
    w[1] = float("nan")
    d = [t.to(dev) for t in (x, dy, w)]
    o = torch.from_numpy(off).to(dev)
    y = _np(_fg8().grouped_gemm_bf16(d[0], d[2], o))
    dx = _np(_fg8().grouped_gemm_bf16_dgrad(d[1], d[2], o))
    dw = _np(_fg8().grouped_gemm_bf16_wgrad(d[1], d[0], o))
    for t in (y, dx):
        assert np.isfinite(np.delete(t, slice(70, 73), 0)).all() and np.isnan(t[70:73]).all()
    assert np.isfinite(dw[[0, 2]]).all() and np.isnan(dw[1]).all()


def test_grouped_offsets_are_clamped(dev):
    """Offsets outside [0, rows] are cut to it; nothing past the tensors is
    touched."""
    g = _gen(6)
    x, w = _bf16(g, 40, 64), _bf16(g, 2, 24, 64)
    off = np.array([-5, 10, 1000], np.int32)
    want, s = layer.grouped(_np(x), _np(w), [0, 10, 40])
    y = _fg8().grouped_gemm_bf16(x.to(dev), w.to(dev), torch.from_numpy(off).to(dev), out_dtype=F32)
    _check(y, want, _sum_error(64, s), "y")
    want, s = layer.grouped_wgrad(_np(x), _np(x), [0, 10, 40])
    dw = _fg8().grouped_gemm_bf16_wgrad(x.to(dev), x.to(dev), torch.from_numpy(off).to(dev))
    _check(dw, want, _sum_error(30, s), "dw")


def test_grouped_no_rows(dev):
    fg8 = _fg8()
    off = torch.zeros(4, dtype=torch.int32, device=dev)
    x, w = torch.empty(0, 64, dtype=BF16, device=dev), torch.zeros(3, 32, 64, dtype=BF16, device=dev)
    dy = torch.empty(0, 32, dtype=BF16, device=dev)
    assert fg8.grouped_gemm_bf16(x, w, off).shape == (0, 32)
    assert fg8.grouped_gemm_bf16_dgrad(dy, w, off).shape == (0, 64)
    dw = torch.full((3, 32, 64), 5.0, device=dev)
    fg8.grouped_gemm_bf16_wgrad(dy, x, off, out=dw)
    assert not dw.any()


def test_grouped_on_another_stream(dev):
    """The call runs on the current stream, with its tensors' work before it."""
    g = _gen(7)
    x, w = _bf16(g, 700, 512).to(dev), _bf16(g, 4, 512, 512).to(dev)
    off = torch.from_numpy(_offsets([100, 250, 50, 300])).to(dev)
    base = _fg8().grouped_gemm_bf16(x, w, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x2 = x * 2
        y2 = _fg8().grouped_gemm_bf16(x2, w, off)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y2, base * 2)


# ---------------------------------------------------------------- dense
# m, n, k: one of each tile, k splits among them, ends inside tiles, odd n
DENSE = [(1, 1, 8), (1, 130, 4096), (7, 37, 40), (16, 64, 512), (33, 70, 1000), (64, 2112, 1024),
         (65, 128, 72), (200, 264, 2048), (300, 515, 136), (4095, 4095, 72)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense_forward(dev, m, n, k, act):
    print(f"dense forward {m}x{n}x{k} {act}", flush=True)
    g = _gen(8, m, n, k)
    x, w = _bf16(g, m, k), _bf16(g, n, k, scale=k ** -0.5)
    bias_type = BF16 if act in ("none", "silu") else F32
    bias, res = torch.randn(n, generator=g).to(bias_type), _bf16(g, m, n)
    z0, s = layer.dense(_np(x), _np(w), _np(bias))
    e = _sum_error(k, s) + 2.0 ** -20 * np.abs(z0)
    a0 = layer.activation(act, z0)
    for with_res in (False, True):
        r = _np(res) if with_res else 0.0
        want = a0 + r
        err = 1.13 * e + 2.0 ** -20 * (np.abs(z0) + np.abs(a0) + np.abs(r))
        out = F32 if with_res else BF16
        y, z = _fg8().gemm_bf16_epilogue(_strided(x, dev, 8), w.to(dev), bias.to(dev),
                                         _strided(res, dev, 3) if with_res else None,
                                         activation=act, save_z=True, out_dtype=out)
        _check(z, z0, e, "z")
        _check(y, want, err, "y")


def test_dense_forward_in_place_of_the_residual(dev):
    g = _gen(9)
    x, w, res = _bf16(g, 50, 256), _bf16(g, 72, 256, scale=1 / 16), _bf16(g, 50, 72)
    z0, s = layer.dense(_np(x), _np(w))
    stream = res.to(dev)
    y = _fg8().gemm_bf16_epilogue(x.to(dev), w.to(dev), residual=stream, out=stream)
    assert y.data_ptr() == stream.data_ptr()
    _check(y, z0 + _np(res), _sum_error(256, s) + 2.0 ** -20 * (np.abs(z0) + np.abs(_np(res))), "y")


def test_dense_forward_twice_gives_the_same_bits(dev):
    """k is split over workgroups here; the parts are added in a fixed order."""
    g = _gen(10)
    x, w = _bf16(g, 40, 7168).to(dev), _bf16(g, 520, 7168).to(dev)
    first = _fg8().gemm_bf16_epilogue(x, w, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(first, _fg8().gemm_bf16_epilogue(x, w, out_dtype=F32))


def test_dense_forward_infinities(dev):
    """exp and erf at the ends of the range: the activations' limits, no NaN
    from finite values."""
    x = torch.zeros(4, 8, dtype=BF16)
    x[:, 0] = torch.tensor([1e30, -1e30, 88.0, -200.0])
    w = torch.zeros(1, 8, dtype=BF16)
    w[0, 0] = 1
    for act in ("relu", "silu", "gelu"):
        y = _np(_fg8().gemm_bf16_epilogue(x.to(dev), w.to(dev), activation=act, out_dtype=F32))[:, 0]
        top = _np(x)[:, 0]
        assert y[0] == top[0] and y[2] == 88.0 and abs(y[1]) == 0 and abs(y[3]) < 1e-30


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 8), (5, 37, 40), (70, 64, 72), (130, 515, 264), (1000, 96, 128),
                                   (513, 520, 1024)])
def test_dense_backward(dev, m, n, k, act):
    print(f"dense backward {m}x{n}x{k} {act}", flush=True)
    g = _gen(11, m, n, k)
    x, w, dy = _bf16(g, m, k), _bf16(g, n, k), _bf16(g, m, n)
    z = _bf16(g, m, n, scale=2.0)
    z[0, 0] = 0.0
    dz = _np(dy) * layer.slope(act, _np(z))
    # dz from the hardware exp and erff (2^-20 of the terms of the slope, each
    # below |z| + 2), then its rounding to BF16
    term = np.abs(_np(dy)) * (np.abs(_np(z)) + 2) * (2.0 ** -20 if act != "none" else 0.0)
    off = term + (2.0 ** -8 * (np.abs(dz) + term) if act != "none" else 0.0)
    want = {"dx": dz @ _np(w), "dw": dz.T @ _np(x), "db": dz.sum(0)}
    err = {"dx": off @ np.abs(_np(w)) + _sum_error(n, (np.abs(dz) + off) @ np.abs(_np(w))),
           "dw": off.T @ np.abs(_np(x)) + _sum_error(m, (np.abs(dz) + off).T @ np.abs(_np(x))),
           "db": term.sum(0) + _sum_error(m, np.abs(dz).sum(0))}
    for dw_dtype in (BF16, F32):
        dx, dw, db = _fg8().gemm_bf16_epilogue_backward(_strided(dy, dev, 3), _strided(x, dev, 8), w.to(dev),
                                                        z.to(dev), activation=act, dw_dtype=dw_dtype)
        _check(dx, want["dx"], err["dx"], "dx")
        _check(dw, want["dw"], err["dw"], "dw")
        _check(db, want["db"], err["db"], "dbias")


def test_dense_backward_only_what_is_needed(dev):
    g = _gen(12)
    x, w, dy = _bf16(g, 96, 64).to(dev), _bf16(g, 40, 64).to(dev), _bf16(g, 96, 40).to(dev)
    full = _fg8().gemm_bf16_epilogue_backward(dy, x, w)
    for i in range(3):
        needs = [j == i for j in range(3)]
        part = _fg8().gemm_bf16_epilogue_backward(dy, x, w, needs=needs)
        assert [p is not None for p in part] == needs and torch.equal(part[i], full[i])


def test_dense_in_a_graph(dev):
    """Captured, replayed several times with eager work in between, every
    replay equal to the eager call (split k: the counters return to zero)."""
    fg8 = _fg8()
    g = _gen(13)
    x, w = _bf16(g, 48, 2048).to(dev), _bf16(g, 200, 2048).to(dev)
    ws = torch.zeros(fg8._lib.lib().fg8_gemm_bf16_workspace_bytes(48, 200, 2048), dtype=torch.uint8, device=dev)
    assert ws.numel() > 0
    out = torch.empty(48, 200, dtype=BF16, device=dev)
    fg8.gemm_bf16_epilogue(x, w, activation="gelu", out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg8.gemm_bf16_epilogue(x, w, activation="gelu", out=out, workspace=ws)
    for i in range(4):
        x.copy_(_bf16(g, 48, 2048).to(dev))
        want = fg8.gemm_bf16_epilogue(x, w, activation="gelu")
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"


def test_dense_backward_of_no_rows(dev):
    x, w, dy = (torch.zeros(0, 64, dtype=BF16, device=dev), torch.ones(40, 64, dtype=BF16, device=dev),
                torch.zeros(0, 40, dtype=BF16, device=dev))
    dx, dw, db = _fg8().gemm_bf16_epilogue_backward(dy, x, w, z=dy, activation="relu")
    assert dx.shape == (0, 64) and not dw.any() and dw.shape == (40, 64) and not db.any() and db.shape == (40,)


def test_dense_backward_relu_stops_infinities(dev):
    """Where z <= 0 nothing passes, whatever dy holds."""
    z = torch.tensor([[-1.0, 0.0, 2.0, -0.0, 3.0]] * 3, dtype=BF16)
    dy = torch.tensor([[float("inf"), float("nan"), 1.0, float("-inf"), -4.0]] * 3, dtype=BF16)
    w = torch.eye(5, 8, dtype=BF16)
    dx, dw, db = _fg8().gemm_bf16_epilogue_backward(dy.to(dev), torch.ones(3, 8, dtype=BF16, device=dev), w.to(dev),
                                                    z=z.to(dev), activation="relu")
    want = np.array([0.0, 0.0, 1.0, 0.0, -4.0])
    assert (_np(dx)[:, :5] == want).all() and (_np(dx)[:, 5:] == 0).all()
    assert (_np(db) == 3 * want).all() and (_np(dw) == 3 * want[:, None]).all()


def test_dense_in_a_graph_with_its_own_workspace(dev):
    """A graph that leaves the workspace to the library stays right when a
    later call of the same stream needs a larger one, and the pass behind it
    (dz and both products) too."""
    fg8 = _fg8()
    g = _gen(14)
    x, w, dy = _bf16(g, 48, 2048).to(dev), _bf16(g, 200, 2048).to(dev), _bf16(g, 48, 200).to(dev)
    assert fg8._lib.lib().fg8_gemm_bf16_workspace_bytes(48, 200, 2048) > 0
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        fg8.gemm_bf16_epilogue(x, w, activation="silu", save_z=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, z = fg8.gemm_bf16_epilogue(x, w, activation="silu", save_z=True)
        grads = fg8.gemm_bf16_epilogue_backward(dy, x, w, z=z, activation="silu")
    for i in range(4):
        x.copy_(_bf16(g, 48, 2048).to(dev))
        want, want_z = fg8.gemm_bf16_epilogue(x, w, activation="silu", save_z=True)
        want_grads = fg8.gemm_bf16_epilogue_backward(dy, x, w, z=want_z, activation="silu")
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            big = [_bf16(g, 64, 4096 * (i + 1)).to(dev) for _ in range(2)]
            fg8.gemm_bf16_epilogue(*big)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want_z), f"replay {i}"
        assert all(torch.equal(a, b) for a, b in zip(grads, want_grads)), f"replay {i}"


# ------------------------------------------------- every tile, at its sizes
def _check_on_gpu(got, want, s, k, what):
    err = _sum_error(k, s)
    if got.dtype == BF16:
        err = err + 2.0 ** -8 * (want.abs() + err)
    bad = ~((got.double() - want).abs() <= err + 1e-38)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off"


# rows a run on average, n, k: thin, flat, low, mid and big tiles (and the
# few-rows kernel) of the forward pass and of the input gradient
@pytest.mark.parametrize("experts,rows,n,k", [(8, 40, 1024, 520), (5, 33, 200, 4360), (6, 150, 1000, 136),
                                              (9, 500, 136, 200), (16, 700, 1032, 1096), (16, 2100, 1096, 1032),
                                              (4, 3000, 4104, 264)])
def test_grouped_tiles(dev, experts, rows, n, k):
    """Float64 products on the GPU as the reference: one product an expert."""
    print(f"grouped tiles {experts} experts {rows} rows {n}x{k}", flush=True)
    g = _gen(14, rows, n)
    cut = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g)).values.tolist()
    off = [0] + cut + [rows]
    x, dy, w = _bf16(g, rows, k).to(dev), _bf16(g, rows, n).to(dev), _bf16(g, experts, n, k).to(dev)
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    y, dx = _fg8().grouped_gemm_bf16(x, w, o), _fg8().grouped_gemm_bf16_dgrad(dy, w, o, out_dtype=F32)
    for e in range(experts):
        a, b = off[e], off[e + 1]
        we = w[e].double()
        _check_on_gpu(y[a:b], x[a:b].double() @ we.T, x[a:b].double().abs() @ we.abs().T, k, f"y of expert {e}")
        _check_on_gpu(dx[a:b], dy[a:b].double() @ we, dy[a:b].double().abs() @ we.abs(), n, f"dx of expert {e}")


# the weight gradient's tiles: 128 x 128; 128 x 256 with 32-deep steps (many
# tiles of short runs); 256 x 256 (long runs)
@pytest.mark.parametrize("experts,rows,n,k", [(5, 700, 520, 264), (40, 900, 1800, 1544), (64, 33000, 2048, 2040)])
def test_grouped_wgrad_tiles(dev, experts, rows, n, k):
    print(f"grouped wgrad tiles {experts} experts {rows} rows {n}x{k}", flush=True)
    g = torch.Generator(device=dev).manual_seed(rows)
    share = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g, device=dev)).values.tolist()
    off = [0] + share + [rows]
    x = torch.randn(rows, k, generator=g, device=dev).to(BF16)
    dy = torch.randn(rows, n, generator=g, device=dev).to(BF16)
    dw = _fg8().grouped_gemm_bf16_wgrad(dy, x, torch.tensor(off, dtype=torch.int32, device=dev))
    for e in range(experts):
        a, b = off[e], off[e + 1]
        p, q = dy[a:b].double().T, x[a:b].double()
        _check_on_gpu(dw[e], p @ q, p.abs() @ q.abs(), b - a, f"dw of expert {e}")


# ---------------------------------------------------------------- refusals
def test_refusals(dev):
    fg8 = _fg8()
    t = lambda *s, d=BF16: torch.zeros(*s, dtype=d, device=dev)   # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises(fg8.Fg8Error, match="multiple of 8"):
        fg8.grouped_gemm_bf16(t(4, 12), t(2, 8, 12), off)
    with pytest.raises(fg8.Fg8Error, match="multiple of 8"):
        fg8.grouped_gemm_bf16_dgrad(t(4, 12), t(2, 12, 8), off)
    with pytest.raises(fg8.Fg8Error, match="ldx"):
        fg8.grouped_gemm_bf16(t(4, 20)[:, :16], t(2, 8, 16), off)
    with pytest.raises(fg8.Fg8Error, match="aligned"):
        fg8.grouped_gemm_bf16(t(4, 32)[:, 4:20], t(2, 8, 16), off)
    with pytest.raises(ValueError, match="disagree"):
        fg8.grouped_gemm_bf16(t(4, 24), t(2, 8, 16), off)
    with pytest.raises(ValueError, match="row_offsets"):
        fg8.grouped_gemm_bf16(t(4, 16), t(3, 8, 16), off)
    with pytest.raises(TypeError, match="x must be"):
        fg8.grouped_gemm_bf16(t(4, 16, d=F32), t(2, 8, 16), off)
    with pytest.raises(ValueError, match="contiguous"):
        fg8.grouped_gemm_bf16(t(16, 4).T, t(2, 8, 16), off)
    with pytest.raises(TypeError, match="output dtype"):
        fg8.grouped_gemm_bf16(t(4, 16), t(2, 8, 16), off, out_dtype=torch.float16)
    with pytest.raises(KeyError):
        fg8.gemm_bf16_epilogue(t(4, 16), t(8, 16), activation="tanh")
    with pytest.raises(ValueError, match="bias"):
        fg8.gemm_bf16_epilogue(t(4, 16), t(8, 16), bias=t(9))
    with pytest.raises(ValueError, match="residual"):
        fg8.gemm_bf16_epilogue(t(4, 16), t(8, 16), residual=t(4, 9))
    with pytest.raises(fg8.Fg8Error, match="workspace"):
        fg8.gemm_bf16_epilogue(t(40, 7168), t(520, 7168), workspace=torch.zeros(64, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError, match="z is needed"):
        fg8.gemm_bf16_epilogue_backward(t(4, 8), t(4, 16), t(8, 16), activation="gelu")
