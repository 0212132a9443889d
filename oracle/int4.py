"""Plain forms of the 4-bit weights with group scales: the quantizer by its
definition, and the values that codes stand for.  No code shared with the HIP
path.
"""
import numpy as np


def bf16(v):
    """The BF16 value nearest to each float32 value, ties to even (finite)."""
    b = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + (b >> np.uint64(16) & np.uint64(1))) & np.uint64(0xFFFF0000)
    return b.astype(np.uint32).view(np.float32)


def quantize(w, group, scales_bf16=False):
    """(codes uint8 [rows, cols], scales float32 [cols / group, rows]) of finite
    float32 w [rows, cols]: s = fl32(amax / 7), 1 where that is 0; code =
    rne(fl32(w / s)) + 8, the quotient limited to -7 .. 7 (a subnormal s may be far
    below amax / 7)."""
    w = np.asarray(w, np.float32)
    rows, cols = w.shape
    codes = np.empty((rows, cols), np.uint8)
    scales = np.empty((cols // group, rows), np.float32)
    for j in range(cols // group):
        part = w[:, j * group:(j + 1) * group]
        s = (np.abs(part).max(1) / np.float32(7)).astype(np.float32)
        if scales_bf16:
            s = bf16(s)
        s = np.where(s == 0, np.float32(1), s)
        codes[:, j * group:(j + 1) * group] = np.rint(np.clip((part / s[:, None]).astype(np.float32), -7, 7)).astype(np.int32) + 8
        scales[j] = s
    return codes, scales


def pack(codes):
    """Column 2 j in the low four bits of byte j."""
    return codes[..., 0::2] | codes[..., 1::2] << 4


def values(codes, scales):
    """float64 values of codes [rows, cols] with scales [cols / group, rows]."""
    group = codes.shape[1] // scales.shape[0]
    return (codes.astype(np.float64) - 8) * np.repeat(np.asarray(scales, np.float64).T, group, 1)
