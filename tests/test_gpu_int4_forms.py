"""Every form of the 4-bit product (rows of x that are copied, weight rows a wave,
waves on k) with every group and type of scales, at odd widths and an odd number of
scales, exactly: with integer x and scales of powers of two every partial sum is an
integer below 2^24 times one power of two."""
import numpy as np
import pytest
import torch

from oracle import int4, layer

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# m, weight rows: one to two rows and three to four, narrow weights and wide ones; up to
# 64 rows, likewise; more
DENSE = [(1, 37), (2, 37), (1, 4101), (2, 4101), (3, 37), (4, 37), (3, 4101), (4, 4101), (5, 71), (16, 71), (33, 8197), (64, 4101), (65, 71), (131, 205)]


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


def _operands(g, sets, m, wide, k, group):
    codes = torch.randint(0, 16, (sets, wide, k), generator=g, dtype=torch.uint8).numpy()
    scales = 2.0 ** torch.randint(-1, 2, (sets, k // group, wide), generator=g).float()
    return codes, scales, torch.randint(-6, 7, (m, k), generator=g).to(BF16)


def _behind(t, dev):
    """t with NaN behind it."""
    room = torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device=dev)
    room[:t.numel()] = t.to(dev).flatten()
    return room[:t.numel()].view(t.shape)


@pytest.mark.parametrize("scales_type", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n", DENSE)
def test_dense(dev, m, n, group, scales_type):
    print(f"int4 {m}x{n} group {group} {scales_type}", flush=True)
    g = torch.Generator().manual_seed(m + 7 * n + group)
    for groups in (1, 3, 11):
        k = groups * group
        codes, scales, x = _operands(g, 1, m, n, k, group)
        y = _fg8().gemm_bf16_int4(x.to(dev), torch.from_numpy(int4.pack(codes[0])).to(dev), _behind(scales[0].to(scales_type), dev), out_dtype=F32)
        want = x.double().numpy() @ int4.values(codes[0], scales[0].numpy()).T
        assert np.array_equal(y.cpu().double().numpy(), want), k


@pytest.mark.parametrize("scales_type", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n", [(1, 37), (4, 2101), (7, 37), (40, 133), (70, 71)])
def test_gated(dev, m, n, group, scales_type):
    """act none: h = z_gate z_up of exact sums, one product rounded to FP32."""
    print(f"int4 gated {m}x{n} group {group} {scales_type}", flush=True)
    g = torch.Generator().manual_seed(m + 5 * n + group)
    for groups in (1, 5):
        k = groups * group
        codes, scales, x = _operands(g, 1, m, 2 * n, k, group)
        h = _fg8().gemm_bf16_int4(x.to(dev), torch.from_numpy(int4.pack(codes[0])).to(dev), _behind(scales[0].to(scales_type), dev), gated=True,
                                  out_dtype=F32)
        z = x.double().numpy() @ int4.values(codes[0], scales[0].numpy()).T
        assert np.array_equal(h.cpu().numpy(), (z[:, :n] * z[:, n:]).astype(np.float32)), k


@pytest.mark.parametrize("scales_type", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts", [[3, 0, 17, 1, 2], [40, 0, 33, 70, 1]])
def test_runs(dev, counts, group, scales_type):
    print(f"int4 runs {counts} group {group} {scales_type}", flush=True)
    g = torch.Generator().manual_seed(sum(counts) + group)
    off = np.concatenate([[1], 1 + np.cumsum(counts)]).astype(np.int32)
    rows, n = int(off[-1]) + 2, 43
    for groups in (1, 3, 11):
        codes, scales, x = _operands(g, len(counts), rows, n, groups * group, group)
        want, _ = layer.grouped(x.double().numpy(), np.stack([int4.values(c, s) for c, s in zip(codes, scales.numpy())]), off)
        x[:1] = x[int(off[-1]):] = float("nan")
        y = _fg8().grouped_gemm_bf16_int4(x.to(dev), torch.from_numpy(int4.pack(codes)).to(dev), _behind(scales.to(scales_type), dev),
                                          torch.from_numpy(off).to(dev), out_dtype=F32)
        assert np.array_equal(y.cpu().double().numpy(), want), groups
