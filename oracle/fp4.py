"""Plain CPU reference of the 4-bit expert weights (NumPy, fp64): E2M1 codes
with one E8M0 scale per 32 weights, from the format's definition.  Test
infrastructure: it shares no code with the HIP path."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])
GROUP = 32


def scale_value(code):
    """2^(code - 127), NaN for 255."""
    code = np.asarray(code).astype(np.int64)
    return np.where(code == 255, np.nan, np.ldexp(1.0, code - 127))


def quantize(w):
    """(codes [.., K], scales [.., K / 32]) of w [.., K], unpacked."""
    w = np.asarray(w, np.float64)
    groups = w.reshape(*w.shape[:-1], -1, GROUP)
    codes = np.zeros(groups.shape, np.uint8)
    scales = np.zeros(groups.shape[:-1], np.uint8)
    for at in np.ndindex(scales.shape):
        v = groups[at]
        most = np.abs(v).max()
        if not np.isfinite(v).all():
            scales[at], step = 255, 1.0
            v = np.zeros(GROUP)  # the codes of such a group mean nothing
        else:
            p = -126
            while most > 7 * 2.0 ** p:
                p += 1
            scales[at], step = p + 127, 2.0 ** p
        a = np.abs(v / step)
        # nearest of the eight magnitudes; of two as near, the one of even code
        d = np.abs(a[:, None] - E2M1[None, :8])
        near = d == d.min(1, keepdims=True)
        code = np.array([min(np.nonzero(n)[0], key=lambda c: (c % 2, c)) for n in near])
        codes[at] = np.where(v < 0, code + 8, code)
    return codes.reshape(w.shape), scales


def dequantize(codes, scales):
    with np.errstate(invalid="ignore"):
        return E2M1[codes] * np.repeat(scale_value(scales), GROUP, axis=-1)


def to_bytes(codes):
    """Two codes per byte, the lower k in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def pack_codes(codes):
    """[.., N, K] codes in fragment order, as bytes [.., N, K / 2]."""
    *lead, N, K = codes.shape
    out = np.zeros((*lead, N // 16, K // 128, 2, 64, 2, 4), np.uint8)
    for lane in range(64):
        r, g = lane % 16, lane // 16
        for s in range(4):
            for b in range(4):
                k = 32 * s + 8 * g + 2 * b
                c = codes.reshape(*lead, N // 16, 16, K // 128, 128)
                out[..., s // 2, lane, s % 2, b] = c[..., r, :, k] | (c[..., r, :, k + 1] << 4)
    return out.reshape(*lead, N, K // 2)


def pack_scales(scales):
    """[.., N, K / 32] scales in fragment order."""
    *lead, N, G = scales.shape
    s = scales.reshape(*lead, N // 16, 16, G // 4, 4)
    return np.ascontiguousarray(np.swapaxes(s, -3, -2)).reshape(*lead, N, G)
