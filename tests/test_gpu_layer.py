"""Layer norm and the MoE combine, forward and backward, against the float64
forms.

Bounds, with u = 2^-24 and C columns.  An FP32 sum of n terms is off by at most
n u times the sum of their absolute values; sqrt, division and each elementary
step add a few u.  Layer norm: the mean is off by e_m = (C + 2) u mean|x|; the
centred values by e_m + u|x|; the variance, relatively, by (C + 4) u plus
2 e_m / sigma; rstd by half of that; y by |h w| times rstd's part plus
(e_m + u |x|) rstd |w| plus a few u of its terms.  The backward pass is bounded
the same way from its two means.  A BF16 output adds 2^-8 relative
(half an ulp, 2^(e-8), of a value of 2^e or more).
"""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _gen(*key):
    return torch.Generator().manual_seed(sum((i + 1) * 104729 * k for i, k in enumerate(key)) + 3)


def _np(t):
    return t.detach().cpu().double().numpy()


def _check(got, want, err, what):
    rounding = 2.0 ** -8 * (np.abs(want) + err) if got.dtype == BF16 else 0.0
    g = _np(got)
    assert g.shape == want.shape
    bad = ~(np.abs(g - want) <= err + rounding + 1e-38)
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} off, first at "
                           f"{np.argwhere(bad)[0]}: {g[bad][0]} for {want[bad][0]}")


def _strided(t, dev, extra):
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=dev)
    wide[:, :t.shape[1]] = t.to(dev)
    return wide[:, :t.shape[1]]


# every team shape, ends inside 16-byte pieces, one row, one column
ROWS_COLS = [(1, 1), (3, 7), (5, 256), (9, 512), (4, 513), (7, 1000), (2, 1025), (300, 1111), (5, 2048),
             (6, 2051), (3, 4096), (5, 4100), (1500, 4104), (2, 7168), (5, 8193), (3, 16384), (2, 16391), (2, 32768)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", ROWS_COLS)
def test_layer_norm(dev, rows, cols, dtype):
    print(f"layer norm {rows}x{cols} {dtype}", flush=True)
    g = _gen(1, rows, cols)
    x = ((torch.randn(rows, cols, generator=g) + 0.5) * torch.exp(torch.randn(rows, 1, generator=g))).to(dtype)
    w_type = BF16 if cols % 2 else F32
    w, b = (1 + 0.1 * torch.randn(cols, generator=g)).to(w_type), torch.randn(cols, generator=g).to(w_type)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    eps = 1e-5
    for bias in (b, None):
        y0, m0, r0 = layer.layer_norm(_np(x), _np(w), None if bias is None else _np(bias), eps)
        y, mean, rstd = _fg8().layer_norm(_strided(x, dev, rows % 3), w.to(dev), None if bias is None else bias.to(dev), eps)
        X = np.abs(_np(x))
        e_m = (cols + 2) * U * X.mean(1)
        sigma = 1 / r0
        e_r = ((cols + 8) * U + 2 * (e_m + U * X.max(1)) / sigma) * r0
        h = (_np(x) - m0[:, None]) * r0[:, None]
        W = np.abs(_np(w))
        e_y = W * (np.abs(h) * (e_r / r0 + 4 * U)[:, None] + ((e_m[:, None] + 2 * U * X) * r0[:, None])) + 4 * U * np.abs(y0)
        e_y += 4 * U * (0 if bias is None else np.abs(_np(bias)))
        _check(mean, m0, e_m, "mean")
        _check(rstd, r0, e_r, "rstd")
        _check(y, y0, e_y, "y")
    # backward, from the saved statistics as they are
    mean, rstd = torch.from_numpy(m0).float(), torch.from_numpy(r0).float()
    dx0, dw0, db0 = layer.layer_norm_backward(_np(dy), _np(x), _np(w), _np(mean), _np(rstd))
    dx, dw, db = _fg8().layer_norm_backward(_strided(dy, dev, rows % 2), _strided(x, dev, rows % 3), w.to(dev), mean.to(dev), rstd.to(dev))
    R, M = _np(rstd)[:, None], np.abs(_np(mean))[:, None]
    h = (_np(x) - _np(mean)[:, None]) * R
    e_h = 3 * U * (np.abs(_np(x)) + M) * R                     # of each h
    G = np.abs(_np(dy)) * W
    H = np.abs(h) + e_h
    e_c1 = (cols + 3) * U * G.mean(1, keepdims=True)
    e_c2 = ((cols + 4) * U * G * H + G * e_h).mean(1, keepdims=True)
    c2 = np.abs((_np(dy) * _np(w) * h).mean(1, keepdims=True))
    e_dx = R * (4 * U * (G + G.mean(1, keepdims=True) + H * (c2 + e_c2)) + e_c1 + H * e_c2 + e_h * c2)
    _check(dx, dx0, e_dx, "dx")
    _check(dw, dw0, ((rows + 3) * U * np.abs(_np(dy)) * H + np.abs(_np(dy)) * e_h).sum(0), "dweight")
    _check(db, db0, ((rows + 2) * U * np.abs(_np(dy))).sum(0), "dbias")


def test_layer_norm_statistics_of_a_far_mean(dev):
    """The variance is taken around the mean: a mean 4096 times the deviation
    does not swallow it (mean x^2 - mean^2 in FP32 would lose it all)."""
    g = _gen(2)
    x = 4096 + torch.randn(8, 1024, generator=g)
    y0, m0, r0 = layer.layer_norm(_np(x), np.ones(1024), None, 0.0)
    y, mean, rstd = _fg8().layer_norm(x.to(dev), torch.ones(1024, device=dev), None, 0.0)
    # the mean's error, at most 1026 u 4096 = 0.25, enters the variance squared
    assert np.abs(_np(rstd) - r0).max() < 0.04 and np.abs(_np(mean) - m0).max() <= 0.26


def test_layer_norm_of_equal_and_broken_rows(dev):
    """A row of one value has no variance: y is the bias.  A row with a NaN or
    an infinity is NaN and leaves the others alone."""
    x = torch.randn(6, 640, generator=_gen(3))
    x[1] = 2.5
    x[2, 600] = float("nan")
    x[4, 0] = float("inf")
    b = torch.randn(640, generator=_gen(4))
    y, _, rstd = _fg8().layer_norm(x.to(dev), torch.ones(640, device=dev), b.to(dev), 1e-5)
    y = y.cpu()
    assert torch.equal(y[1], b) and abs(float(rstd[1]) - 1e-5 ** -0.5) < 1e-4 * 1e-5 ** -0.5
    assert y[2].isnan().all() and y[4].isnan().all() and y[[0, 1, 3, 5]].isfinite().all()


def test_layer_norm_shapes_and_no_rows(dev):
    fg8 = _fg8()
    w = torch.ones(96, device=dev)
    x = torch.randn(2, 3, 96, generator=_gen(5)).to(dev)
    y, mean, rstd = fg8.layer_norm(x, w)
    flat = fg8.layer_norm(x.reshape(6, 96), w)
    assert y.shape == x.shape and mean.shape == (2, 3) and torch.equal(y.reshape(6, 96), flat[0])
    dx, dw, db = fg8.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == x.shape
    none = torch.empty(0, 96, device=dev)
    assert fg8.layer_norm(none, w)[0].shape == (0, 96)
    dx, dw, db = fg8.layer_norm_backward(none, none, w, mean[:0, 0].contiguous(), rstd[:0, 0].contiguous())
    assert dx.shape == (0, 96) and not dw.any() and not db.any()


def test_layer_norm_gradient_against_differences(dev):
    """The kernel's own forward pass, differenced: with step 2^-6 along v the
    third-order term is below 1e-3 of the slope and the FP32 noise of the two
    losses (about sqrt(n) u sum|terms| / step) below 1e-3 too."""
    fg8 = _fg8()
    g = _gen(6)
    x, v, w, dy = (torch.randn(16, 384, generator=g).to(dev) for _ in range(4))
    w = w[0].contiguous()
    _, mean, rstd = fg8.layer_norm(x, w)
    dx, _, _ = fg8.layer_norm_backward(dy, x, w, mean, rstd)
    h = 2.0 ** -6
    loss = lambda a: (dy.double() * fg8.layer_norm(a, w)[0].double()).sum()   # noqa: E731
    slope = float((loss(x + h * v) - loss(x - h * v)) / (2 * h))
    want = float((dx.double() * v.double()).sum())
    scale = float((dx.double().norm() * v.double().norm()))
    assert abs(slope - want) <= 2e-3 * scale


def test_layer_norm_is_repeatable(dev):
    fg8 = _fg8()
    g = _gen(7)
    x, dy = torch.randn(3000, 520, generator=g).to(dev), torch.randn(3000, 520, generator=g).to(dev)
    w = torch.ones(520, device=dev)
    _, mean, rstd = fg8.layer_norm(x, w)
    first = fg8.layer_norm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, fg8.layer_norm_backward(dy, x, w, mean, rstd)))


# ------------------------------------------------------------------ combine
def _maps(g, tokens, topk, rows, dead):
    """token_row and its inverse: each position a row of its own, a share of
    the positions routed nowhere."""
    perm = torch.randperm(rows, generator=g)[:tokens * topk].to(torch.int32)
    perm[torch.rand(tokens * topk, generator=g) < dead] = -1
    row_token = torch.full((rows,), -1, dtype=torch.int32)
    live = perm >= 0
    row_token[perm[live].long()] = (torch.arange(tokens * topk)[live] // topk).to(torch.int32)
    return perm.reshape(tokens, topk), row_token


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,topk,hidden,extra,dead", [
    (1, 1, 8, 0, 0.0), (3, 2, 40, 5, 0.3), (5, 8, 520, 3, 0.1), (17, 7, 1000, 11, 0.5),
    (2, 9, 2048, 1, 0.2), (3, 70, 264, 2, 0.4), (65, 3, 7168, 61, 0.1), (4, 8, 64, 4, 1.0)])
def test_combine(dev, tokens, topk, hidden, extra, dead, dtype):
    print(f"combine {tokens}x{topk}x{hidden} {dtype}", flush=True)
    g = _gen(8, tokens, topk, hidden)
    rows = tokens * topk + extra
    token_row, row_token = _maps(g, tokens, topk, rows, dead)
    y = torch.randn(rows, hidden, generator=g).to(dtype)
    y[row_token < 0] = float("nan")                       # rows that hold no token are not read
    p, res = torch.randn(tokens, topk, generator=g), torch.randn(tokens, hidden, generator=g).to(dtype)
    if dead:
        p[token_row < 0] = float("inf")                   # nor are the weights of dead positions
    dout = torch.randn(tokens, hidden, generator=g).to(dtype)
    clean_y, clean_p = np.nan_to_num(_np(y)), np.where(token_row.numpy() < 0, 0, _np(p))
    at = token_row.numpy()
    d = [t.to(dev) for t in (y, token_row, p, res, dout, row_token)]
    size = layer.combine(np.abs(clean_y), at, np.abs(clean_p))
    for residual in (None, d[3]):
        want = layer.combine(clean_y, at, clean_p, None if residual is None else _np(res))
        # topk products and additions, and the residual's
        err = (topk + 2) * U * (size + (0 if residual is None else np.abs(_np(res))))
        _check(_fg8().moe_combine(d[0], d[1], d[2], residual=residual), want, err, "out")
    dy0, dp0 = layer.combine_backward(_np(dout), clean_y, at, clean_p)
    _, s = layer.combine_backward(np.abs(_np(dout)), np.abs(clean_y), at, np.abs(clean_p))
    dy, dp = _fg8().moe_combine_backward(d[4], d[0], d[1], d[5], d[2])
    _check(dy, dy0, U * np.abs(dy0), "dy")
    _check(dp, dp0, (hidden + 1) * U * s, "dweights")


def test_combine_indices_out_of_range(dev):
    """Positions past the last row add nothing; no memory outside y is read or
    written."""
    fg8 = _fg8()
    y = torch.ones(8, 16, device=dev)
    at = torch.tensor([[0, 8], [2 ** 31 - 1, 3], [-7, 1 << 20]], dtype=torch.int32, device=dev)
    owner = torch.tensor([0, -1, 9, 1, -1, -1, 3, -1], dtype=torch.int32, device=dev)
    p = torch.full((3, 2), 2.0, device=dev)
    out = fg8.moe_combine(y, at, p)
    assert out[:, 0].tolist() == [2.0, 2.0, 0.0]
    dy, dp = fg8.moe_combine_backward(torch.ones(3, 16, device=dev), y, at, owner, p)
    assert dp.tolist() == [[16.0, 0.0], [0.0, 16.0], [0.0, 0.0]]
    assert dy[:, 0].tolist() == [2.0, 0.0, 0.0, 2.0, 0.0, 0.0, 0.0, 0.0]


def test_combine_no_tokens(dev):
    fg8 = _fg8()
    y = torch.ones(8, 16, device=dev)
    at, p = torch.empty(0, 2, dtype=torch.int32, device=dev), torch.empty(0, 2, device=dev)
    assert fg8.moe_combine(y, at, p).shape == (0, 16)
    owner = torch.full((8,), -1, dtype=torch.int32, device=dev)
    dy, dp = fg8.moe_combine_backward(torch.empty(0, 16, device=dev), y, at, owner, p)
    assert not dy.any() and dp.shape == (0, 2)


def test_combine_takes_the_routing_steps_maps(dev):
    fg8 = _fg8()
    g = _gen(9)
    ids = torch.stack([torch.randperm(8, generator=g)[:3] for _ in range(200)]).to(torch.int32)
    ids[::7, 1] = ids[::7, 0]                             # repeats route nowhere
    x = torch.randn(200, 128, generator=g)
    lay = fg8.moe_contiguous_layout_fp8(x.to(dev), ids.to(dev), 8)
    rows = lay["q"].shape[0]
    y = torch.randn(rows, 128, generator=g)
    p = torch.rand(200, 3, generator=g)
    at = lay["token_row"].cpu().numpy()
    out = fg8.moe_combine(y.to(dev), lay["token_row"], p.to(dev))
    want = layer.combine(_np(y), at, _np(p))
    _check(out, want, 5 * U * layer.combine(np.abs(_np(y)), at, _np(p)), "out")
    dy, dp = fg8.moe_combine_backward(x.to(dev), y.to(dev), lay["token_row"], lay["row_token"], p.to(dev))
    dy0, dp0 = layer.combine_backward(_np(x), _np(y), at, _np(p))
    _check(dy, dy0, U * np.abs(dy0), "dy")
    _check(dp, dp0, 129 * U * layer.combine_backward(np.abs(_np(x)), np.abs(_np(y)), at, _np(p))[1], "dweights")


def test_refusals(dev):
    fg8 = _fg8()
    x, w = torch.zeros(4, 64, device=dev), torch.ones(64, device=dev)
    with pytest.raises(TypeError, match="x must be"):
        fg8.layer_norm(x.half(), w)
    with pytest.raises(ValueError, match="weight"):
        fg8.layer_norm(x, w[:32])
    with pytest.raises(TypeError, match="one type"):
        fg8.layer_norm(x, w, w.to(BF16))
    with pytest.raises(fg8.Fg8Error, match="eps"):
        fg8.layer_norm(x, w, eps=-1.0)
    with pytest.raises(fg8.Fg8Error, match="exceeds"):
        fg8.layer_norm(torch.zeros(1, 32769, device=dev), torch.ones(32769, device=dev))
    with pytest.raises(ValueError, match="contiguous"):
        fg8.layer_norm(torch.zeros(64, 4, device=dev).T, w)
    with pytest.raises(ValueError, match="disagree"):
        fg8.layer_norm_backward(x[:3], x, w, w[:4], w[:4])
    at, p = torch.zeros(4, 2, dtype=torch.int32, device=dev), torch.zeros(4, 2, device=dev)
    with pytest.raises(fg8.Fg8Error, match="multiple of 8"):
        fg8.moe_combine(torch.zeros(8, 12, device=dev), at, p)
    with pytest.raises(ValueError, match="token_row"):
        fg8.moe_combine(x, at, p[:3])
    with pytest.raises(ValueError, match="residual"):
        fg8.moe_combine(x, at, p, residual=x[:2])
