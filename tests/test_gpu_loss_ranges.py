"""dx of the loss's backward pass where its sums over the classes are cut into
ranges that are added at the end, and the vocabulary into pieces: against float64
products on the GPU, every element of dx and dw.

Bounds, with u = 2^-24: a logit is off by e = 2 (K + 1) u S, S the sum of the
absolute products; a probability by a factor of e^(e + 2^-17), so dl by (e + 2^-17)
(p + 2^-22) |dloss| + 2^-22 |dl|, and by 2^-8 of itself for its rounding to BF16 (2^-15
in two parts); the sums over V classes or M rows by 2 (V + 1) u or 2 (M + 1) u of
their absolute terms (twice that for two parts), in whatever order and ranges; a
BF16 output by 2^-8 of itself.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _close(got, want, err, what):
    if got.dtype == BF16:
        err = err + 2.0 ** -8 * (want.abs() + err)
    bad = ~((got.double() - want).abs() <= err + 1e-38)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


# m, vocab, k, ranges of a piece's classes (0: none, its sums are the product's own and
# the next piece's are added onto them, in small tiles or big ones), whether there is
# more than one piece: ragged rows, columns and ranges, several column tiles, rows more
# than a piece has classes
CASES = [(2001, 4003, 2056, 3, False), (385, 8197, 4104, 7, False), (4100, 66001, 520, 5, True), (1100, 5001, 1800, 4, False),
         (9000, 40003, 264, 7, True),
         (601, 450001, 72, 0, True), (4090, 70001, 4096, 0, True), (20011, 16411, 72, 3, True)]


@pytest.mark.parametrize("m,v,k,ranges,pieces", CASES)
def test_ranges_and_pieces(dev, m, v, k, ranges, pieces):
    print(f"loss backward {m}x{v}x{k}, {ranges} ranges", flush=True)
    fg8 = _fg8()
    c = fg8.bf16_tile_choice("linear_cross_entropy_dx", m, v, k)
    assert (2 * m * v > 512 << 20) == pieces
    if ranges:
        assert c["splits"] == ranges and c["persistent"]
    else:                    # (a big tile without ranges, or a small one in splits of its own)
        assert c["persistent"] == (m > 1000) and (c["splits"] > 1) == (m < 1000)
    g = torch.Generator(device=dev).manual_seed(m + v)
    x = torch.randn(m, k, device=dev, generator=g).to(BF16)
    w = (torch.randn(v, k, device=dev, generator=g) * 2 * k ** -0.5).to(BF16)
    t = torch.randint(0, v, (m,), device=dev, generator=g)
    t[::7] = -1
    live = t >= 0
    dloss = 0.5 + torch.rand(m, device=dev, generator=g)
    xd, wd = x.double(), w.double()
    l = xd @ wd.T.contiguous()
    lse = torch.logsumexp(l, 1).float()
    clean = torch.where(live, dloss, 0.0).double()[:, None]
    dloss[~live] = float("nan")
    rows = torch.arange(m, device=dev)
    # dx and dw of either type, on the library's workspace and on one that held NaN
    size = fg8._lib.lib().fg8_linear_cross_entropy_backward_workspace_bytes(m, v, k, fg8._lib.OUT_F32)
    poison = torch.full((-(-size // 4),), float("nan"), device=dev)
    poison[:1024] = 0
    dx, dw = fg8.linear_cross_entropy_backward(dloss, x, w, t, lse, dw_dtype=BF16)
    dx32, dw32 = fg8.linear_cross_entropy_backward(dloss, x, w, t, lse, workspace=poison)
    assert torch.equal(dx, dx32)
    del poison
    # (pieces of the classes at a time: dx's sums and bounds are added up)
    dx0, dx_err, dx_size = (torch.zeros(m, k, dtype=F64, device=dev) for _ in range(3))
    for a in range(0, v, 16384):
        b = min(a + 16384, v)
        e = 2 * (k + 1) * U * (xd.abs() @ wd[a:b].abs().T.contiguous())
        p = torch.exp(l[:, a:b] - lse.double()[:, None]) * live[:, None]
        dl = p.clone()
        here = (t >= a) & (t < b)
        dl[rows[here], t[here] - a] -= 1.0
        dl *= clean
        ed = (e + 2.0 ** -17) * (p + 2.0 ** -22) * clean + 2.0 ** -22 * dl.abs()
        r8, r15 = ed + 2.0 ** -8 * (dl.abs() + ed), ed + 2.0 ** -15 * (dl.abs() + ed)
        dx0 += dl @ wd[a:b]
        dx_err += r8 @ wd[a:b].abs()
        dx_size += (dl.abs() + r8) @ wd[a:b].abs()
        want = dl.T.contiguous() @ xd
        for got, r, parts in ((dw, r8, 1), (dw32, r15, 2)):
            size = (dl.abs() + r).T.contiguous() @ xd.abs()
            _close(got[a:b], want, r.T.contiguous() @ xd.abs() + parts * 2 * (m + 1) * U * size, f"dw in {got.dtype}, classes {a} .. {b - 1}")
    _close(dx, dx0, dx_err + 2 * (v + 1) * U * dx_size, "dx")
