"""The cross entropy of a linear head, forward and backward, against float64.

Bounds.  A logit is a sum of K products of BF16 values: off by e = 2 (K + 1) 2^-24 S
at most (S the sum of the absolute products).  lse moves by no more than its
largest logit's error; the exponentials' arguments (l - max) log2 e are off by
2^-23 of at most 60 where they count, and the sum, in any order, by (V + 8) 2^-24:
E = max_c e + 2^-17 + (V + 8) 2^-24 + 2^-23 |lse|.  The loss is off by that, the target's e
and 2^-22 of both logits.  Backward a probability is off by a factor of e^(e + 2^-17)
(its argument, as above), hence dl by (e + 2^-17) (p + 2^-22) |dloss| + 2^-22 |dl|, and 2^-8
of dl for its rounding to BF16 (2^-15 in two parts); the products follow with sums
of their own.
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
    return torch.Generator().manual_seed(sum((i + 1) * 3571 * k for i, k in enumerate(key)) + 17)


def _np(t):
    return t.detach().cpu().double().numpy()


def _sum_error(k, s):
    return 2 * (k + 1) * 2.0 ** -24 * s


def _inputs(case, m, v, k):
    g = _gen(case, m, v)
    x = torch.randn(m, k, generator=g).to(BF16)
    w = (torch.randn(v, k, generator=g) * 3 * k ** -0.5).to(BF16)
    t = torch.randint(0, v, (m,), generator=g)
    t[::5] = -100
    if m > 7:
        t[3], t[6] = v, v - 1         # past the last class; the last class
    return x, w, t


# m, vocab, k: one row, one class, odd vocabularies, every tile, products in several k ranges
CASES = [(1, 1, 8), (1, 1000, 64), (2, 77, 200), (13, 129, 72), (64, 300, 136), (65, 513, 64), (130, 1001, 328), (257, 40, 512), (500, 4099, 72),
         (1100, 8200, 64), (53, 300, 2048), (3, 1158, 4104), (130, 520, 4096), (200, 2000, 2120)]


def _close(got, want, err, what):
    g = _np(got)
    rounding = 2.0 ** -8 * (np.abs(want) + err) if got.dtype == BF16 else 0.0
    bad = ~(np.abs(g - want) <= err + rounding + 1e-38)
    assert not bad.any(), (f"{what}: {np.count_nonzero(bad)} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} for {want[bad][0]}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(dev, case, wide):
    m, v, k = CASES[case]
    print(f"loss {m}x{v}x{k} int64 {wide}", flush=True)
    x, w, t = _inputs(case, m, v, k)
    l, s = layer.dense(_np(x), _np(w))
    e = _sum_error(k, s)
    want, lse = layer.cross_entropy(l, t.numpy())
    big = torch.full((m, k + 8), float("nan"), dtype=BF16, device=dev)
    big[:, :k] = x.to(dev)
    loss, got = _fg8().linear_cross_entropy(big[:, :k], w.to(dev), t.to(torch.int64 if wide else torch.int32).to(dev))
    E = e.max(1) + 2.0 ** -17 + (v + 8) * 2.0 ** -24 + 2.0 ** -23 * np.abs(lse)
    _close(got, lse, E, "lse")
    live = ((t >= 0) & (t < v)).numpy()
    at = np.where(live, t.numpy(), 0)
    rows = np.arange(m)
    _close(loss, want, live * (E + e[rows, at] + 2.0 ** -22 * (np.abs(lse) + np.abs(l[rows, at]))), "loss")


@pytest.mark.parametrize("dw_dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward(dev, case, dw_dtype):
    m, v, k = CASES[case]
    print(f"loss backward {m}x{v}x{k} {dw_dtype}", flush=True)
    x, w, t = _inputs(case, m, v, k)
    l, s = layer.dense(_np(x), _np(w))
    lse = torch.from_numpy(layer.cross_entropy(l, t.numpy())[1]).float()
    dloss = 0.5 + torch.rand(m, generator=_gen(case))
    dloss[::5] = float("nan")                      # rows without a target
    live = ((t >= 0) & (t < v)).numpy()
    clean = torch.where(torch.from_numpy(live), dloss, 0.0)
    dl = layer.cross_entropy_backward(_np(clean), l, t.numpy(), _np(lse))
    p = np.exp(l - _np(lse)[:, None]) * live[:, None]
    ed = (_sum_error(k, s) + 2.0 ** -17) * (p + 2.0 ** -22 * live[:, None]) * _np(clean)[:, None] + 2.0 ** -22 * np.abs(dl)
    ed8, ed15 = ed + 2.0 ** -8 * (np.abs(dl) + ed), ed + 2.0 ** -15 * (np.abs(dl) + ed)
    dx, dw = _fg8().linear_cross_entropy_backward(dloss.to(dev), x.to(dev), w.to(dev), t.to(dev), lse.to(dev), dw_dtype=dw_dtype)
    size, ax, aw = np.abs(dl) + ed8, np.abs(_np(x)), np.abs(_np(w))
    _close(dx, dl @ _np(w), ed8 @ aw + _sum_error(v, size @ aw), "dx")
    e = (ed8 if dw_dtype == BF16 else ed15).T @ ax + (1 if dw_dtype == BF16 else 2) * _sum_error(m, size.T @ ax)
    _close(dw, dl.T @ _np(x), e, "dw")


def test_pieces_of_the_vocabulary(dev):
    """A head whose logits' gradients are more than one piece (of 512 MB): the
    same as the rows on their own, which are one piece, for dx in float sums; and
    dw against float32 products of torch's own logits on sampled classes.

    dx: both sums of V products of the same BF16 factors, in another order and
    rounded once: 2^-8 and 2 (V + 1) 2^-24 of the absolute sums.  dw: ditto with the
    logits' error e (probabilities by a factor e^(e + 2^-17)), 2 * 2^-8 together."""
    m, v, k = 9000, 40003, 64
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(m, k, device=dev, generator=g).to(BF16)
    w = (torch.randn(v, k, device=dev, generator=g) * 0.3).to(BF16)
    t = torch.randint(0, v, (m,), device=dev, generator=g)
    fg8 = _fg8()
    assert 2 * m * v > 512 << 20
    loss, lse = fg8.linear_cross_entropy(x, w, t)
    dloss = torch.rand(m, device=dev, generator=g)
    dx, dw = fg8.linear_cross_entropy_backward(dloss, x, w, t, lse, dw_dtype=BF16)
    some = torch.arange(7, m, 1201, device=dev)
    part, _ = fg8.linear_cross_entropy_backward(dloss[some].contiguous(), x[some], w, t[some], lse[some].contiguous(), needs=(True, False))
    l = x[some].float() @ w.float().T
    dl = torch.exp(l - lse[some][:, None])
    dl[torch.arange(len(some)), t[some]] -= 1
    size = (dl.abs() * dloss[some][:, None]) @ w.float().abs()
    off = (dx[some].float() - part.float()).abs()
    assert (off <= (2.0 ** -8 + 2 * (v + 1) * 2.0 ** -24) * size + 2.0 ** -8 * part.float().abs()).all()
    classes = torch.tensor([0, 255, 256, 19999, 20223, 20224, 20225, 39999, v - 1], device=dev)
    dl = torch.exp(x.float() @ w[classes].float().T - lse[:, None]) - (t[:, None] == classes).float()
    dl *= dloss[:, None]
    want, size = dl.T @ x.float(), dl.abs().T @ x.float().abs()
    assert ((dw[classes].float() - want).abs() <= (2 * 2.0 ** -8 + 2 * (m + 1) * 2.0 ** -24) * size).all()
    wide, dwf = fg8.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.equal(wide, dx)
    assert ((dwf[classes] - want).abs() <= (2.0 ** -13 + 2 * (m + 1) * 2.0 ** -24) * size).all()


@pytest.mark.parametrize("m,v,k", [(33, 70, 72), (70, 33, 2056)])
def test_float_weight_gradient_of_strided_rows(dev, m, v, k):
    """Rows a stride apart, no more of them than classes and more: as laid close."""
    x, w, t = _inputs(60, m, v, k)
    wide = torch.full((m, k + 24), float("nan"), dtype=BF16)
    wide[:, 8:8 + k] = x
    fg8 = _fg8()
    w, t, dloss = w.to(dev), t.to(dev), torch.rand(m, generator=_gen(60)).to(dev)
    _, lse = fg8.linear_cross_entropy(x.to(dev), w, t)
    for a, b in zip(*(fg8.linear_cross_entropy_backward(dloss, r, w, t, lse) for r in (x.to(dev), wide.to(dev)[:, 8:8 + k]))):
        assert torch.equal(a, b) and a.isfinite().all()


def test_against_differences(dev):
    """The mean loss along a direction, by central differences: a relative error
    of the step's square (2^-8) and the gradients' BF16 rounding: 0.02 of the
    gradient's length times the direction's."""
    m, v, k = 40, 200, 64
    x, w, t = _inputs(50, m, v, k)
    fg8 = _fg8()
    count = int(((t >= 0) & (t < v)).sum())

    def value(a, b):
        return float(fg8.linear_cross_entropy(a.to(dev), b.to(dev), t.to(dev))[0].double().sum()) / count
    _, lse = fg8.linear_cross_entropy(x.to(dev), w.to(dev), t.to(dev))
    dx, dw = fg8.linear_cross_entropy_backward(torch.full((m,), 1.0 / count, device=dev), x.to(dev), w.to(dev), t.to(dev), lse)
    for a, grad, is_x in ((x, dx, True), (w, dw, False)):
        d = torch.randn(a.shape, generator=_gen(is_x)) * float(a.float().std()) / 16
        lo, hi = (a.float() - d).to(BF16), (a.float() + d).to(BF16)
        step = hi.double() - lo.double()
        diff = value(hi, w) - value(lo, w) if is_x else value(x, hi) - value(x, lo)
        assert abs(diff - float((grad.cpu().double() * step).sum())) <= 0.02 * float(grad.cpu().double().norm() * step.norm())


def test_extremes(dev):
    """Logits of +-3e4 and rows of equal ones: exact; -inf adds nothing; +inf and
    NaN stay in their rows."""
    fg8 = _fg8()
    v = 300
    w = torch.zeros(v, 8, dtype=BF16)
    w[:, 0] = torch.arange(v) % 3 - 1                 # -1, 0, 1
    w[7, 1] = float("-inf")
    x = torch.zeros(5, 8, dtype=BF16)
    x[0, 0], x[1, 0], x[3, 0], x[4, 0] = 30000, -30000, float("nan"), float("inf")
    x[:, 1] = 0
    x[2, 1] = 1                                       # its logit of class 7 is -inf
    t = torch.tensor([2, 0, 9, 1, 1])
    w2 = w.clone()
    w2[7, 1] = 0                                      # (0 times -inf is NaN: rows 0 and 1 without it)
    big = float(torch.tensor(30000.0).to(BF16))
    loss, lse = fg8.linear_cross_entropy(x.to(dev), w2.to(dev), t.to(dev))
    assert torch.allclose(lse[:2].cpu(), torch.tensor([big, big]) + np.log(100), rtol=2.0 ** -22)
    assert torch.allclose(loss[:2].cpu(), torch.full((2,), np.log(100)), rtol=2.0 ** -20)
    assert torch.allclose(lse[2].cpu(), torch.tensor(np.log(300.0)).float(), rtol=2.0 ** -20)
    assert lse[3:].isnan().all() and loss[3:].isnan().all()
    loss, lse = fg8.linear_cross_entropy(x[2:3].contiguous().to(dev), w.to(dev), t[2:3].to(dev))
    assert torch.allclose(lse.cpu(), torch.tensor([np.log(299.0)]).float(), rtol=2.0 ** -20)
    assert torch.allclose(loss, lse)
    dx, dw = fg8.linear_cross_entropy_backward(torch.ones(5, device=dev), x.to(dev), w2.to(dev), torch.full((5,), -1, device=dev),
                                               torch.zeros(5, device=dev))
    assert not dx.any()                               # no row has a target: x's NaN does not matter to dx


def test_empty_and_needs(dev):
    fg8 = _fg8()
    w = torch.ones(40, 64, dtype=BF16, device=dev)
    loss, lse = fg8.linear_cross_entropy(torch.empty(0, 64, dtype=BF16, device=dev), w, torch.empty(0, dtype=torch.int64, device=dev))
    assert loss.shape == lse.shape == (0,)
    x, t = torch.ones(3, 64, dtype=BF16, device=dev), torch.tensor([1, 2, 3], device=dev)
    loss, lse = fg8.linear_cross_entropy(x, w, t)
    both = fg8.linear_cross_entropy_backward(loss, x, w, t, lse)
    for needs in ((True, False), (False, True)):
        one = fg8.linear_cross_entropy_backward(loss, x, w, t, lse, needs=needs)
        for a, b, n in zip(one, both, needs):
            assert torch.equal(a, b) if n else a is None
    dx, dw = fg8.linear_cross_entropy_backward(loss[:0], x[:0], w, t[:0], lse[:0])
    assert dx.shape == (0, 64) and not dw.any()


def test_captured(dev):
    fg8 = _fg8()
    x, w, t = (a.to(dev) for a in _inputs(60, 70, 1500, 520))

    def both():
        loss, lse = fg8.linear_cross_entropy(x, w, t)
        return (loss, lse, *fg8.linear_cross_entropy_backward(loss, x, w, t, lse))
    want = both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(4):
        for a in got:
            a.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
