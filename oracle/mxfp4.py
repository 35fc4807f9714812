"""MXFP4 -- oracle side: microscaled 4-bit floating point per 32-element block.

The block length is the rotation's.  One scale 2^(s - 127) per block, stored as the
byte s (255 = NaN), and 4-bit e2m1 codes: bit 3 the sign, bits 2..1 the exponent p,
bit 0 the mantissa f; the magnitude is f / 2 for p = 0 and (1 + f / 2) 2^(p - 1)
otherwise: 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Element 2i is the low nibble of byte i.

Quantiser, on the fp32 (optionally rotated) values y of a block: a = max |y|;
E = clamp(floor(log2 a) - 2, -127, 127), -127 when a = 0; s = E + 127; each code is
the e2m1 value nearest to y 2^-E (an exact scaling), ties to the code with f = 0,
magnitudes past 6 to 6.  A block with an infinity or a NaN: s = 255, codes 0.
"""
from __future__ import annotations

import numpy as np

from .hadamard import rotate_h32

#: magnitudes of the e2m1 codes 0..7
E2M1 = np.array([f / 2 if p == 0 else (1 + f / 2) * 2.0 ** (p - 1) for p in range(4) for f in range(2)])


def e2m1_code(v: np.ndarray) -> np.ndarray:
    """Code (uint8 0..15) of the e2m1 value nearest to each finite v; ties to even, saturating."""
    v = np.asarray(v, dtype=np.float64)
    m = np.minimum(np.abs(v), 6.0)
    gap = np.abs(m[..., None] - E2M1)
    best = gap.min(axis=-1, keepdims=True)
    # of the (at most two) nearest codes the even one
    odd_last = np.where(gap == best, np.arange(8) + 8 * (np.arange(8) % 2), 99)
    mag = odd_last.min(axis=-1) % 8
    return (mag + 8 * np.signbit(v)).astype(np.uint8)


def quantize_mxfp4(x: np.ndarray, rotate: bool = True) -> dict:
    """Rows x [rows][K] (fp32 values) -> packed codes [rows][K/2], scale bytes [rows][K/32], unpacked codes."""
    xf = np.asarray(x, dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        y = rotate_h32(xf) if rotate else xf
    rows, K = y.shape
    b = y.reshape(rows, K // 32, 32).astype(np.float64)
    bad = ~np.isfinite(b).all(axis=-1)
    b = np.where(bad[..., None], 0.0, b)
    a = np.abs(b).max(axis=-1)
    with np.errstate(divide="ignore"):
        e = np.where(a > 0, np.clip(np.frexp(a)[1] - 3, -127, 127), -127)  # a = m 2^e, m in [0.5, 1)
    q = e2m1_code(b * np.exp2(-e.astype(np.float64))[..., None])
    q = np.where(bad[..., None], 0, q).reshape(rows, K).astype(np.uint8)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return {"codes": (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8), "scales": s, "q": q, "rotated": bool(rotate)}


def mxfp4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The fp64 values [rows][K] that packed codes and scale bytes stand for."""
    codes = np.asarray(codes, dtype=np.uint8)
    q = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[0], -1)
    v = np.where(q >= 8, -1.0, 1.0) * E2M1[q & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def mxfp4_matmul(w: dict, a: dict) -> np.ndarray:
    """Y[m][n] in fp64 from the codes and scales of weights w [N][K] and activations a [M][K]."""
    return mxfp4_values(a["codes"], a["scales"]) @ mxfp4_values(w["codes"], w["scales"]).T
