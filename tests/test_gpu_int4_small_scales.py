"""The 4-bit quantizer where amax / 7 lies among the subnormals of the scales'
type: a scale of a few bits may be far below it, and the quotient is limited to
what a code holds.

What is asked of a group follows from the definition alone: codes in 1 .. 15; no
sign turned; and a weight off by half a scale at most, or by what it exceeds seven
scales (1 for a scale that rounds to 0, where every code is 8).
"""
import numpy as np
import pytest
import torch

from oracle import int4

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _fg8():
    import moe_grouped_gemm_fp8_amd as fg8
    return fg8


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("source,scales,unit", [(F32, F32, -149), (F32, F32, -147), (F32, BF16, -133), (BF16, BF16, -133), (BF16, F32, -133),
                                                (F32, BF16, -149)])
def test_few_bits(dev, group, source, scales, unit):
    """One row for each largest weight of 1 .. 60 units, other groups beside it."""
    print(f"int4 subnormal scales group {group} {source} {scales} 2^{unit}", flush=True)
    g = torch.Generator().manual_seed(group + unit)
    tops = torch.arange(1, 61)
    w = torch.randn(60, 2 * group, generator=g)                       # (the second group's weights are ordinary)
    few = torch.randint(-60, 61, (60, group), generator=g)
    few = few.clamp(-tops[:, None], tops[:, None])
    few[:, 0], few[:, 1] = tops, -tops
    w[:, :group] = few.float() * 2.0 ** unit
    w = w.to(source)
    assert torch.equal(w[:, :group].double(), few.double() * 2.0 ** unit)
    q, s = _fg8().int4_quantize(w.to(dev), group=group, scale_dtype=scales)
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).cpu().int()
    assert codes.min() >= 1 and codes.max() <= 15
    v = _fg8().int4_dequantize(q, s, out_dtype=F32).cpu().double()[:, :group]
    want, sd = w[:, :group].double(), s[0].cpu().double()[:, None]
    assert (v * want >= 0).all(), "a sign turned"
    assert ((v - want).abs() <= torch.maximum(sd / 2, want.abs() - 7 * sd)).all()
    oracle_codes, oracle_scales = int4.quantize(w.float().numpy(), group, scales == BF16)
    assert np.array_equal(s.float().cpu().numpy(), oracle_scales) and np.array_equal(codes.numpy(), oracle_codes)
