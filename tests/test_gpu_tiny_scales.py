"""int4 and int8 blocks whose scale d is below fp32's normal range but has a finite reciprocal (d > 2^-128): the
fused quantisers round them as the plain ones do.

A read-back value lies within half a step of y.  Beside it: y's fp32 error, 30 u = 30 x 2^-24 of it (the bound of
tests/test_gpu_fused_quant.py for SwiGLU) and its own rounding below the normal range, 2^-150; the stored d and the
value read back are rounded there as well, code x 2^-150 + 2^-150; and the step that the codes were rounded with is
1/d of the rounded d, 2^-150 / 2^-128 = 2^-22 of the value and 2^-24 twice for the reciprocal and the product.
"""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
FMT = {"int4": (7, w4.w4a4_swiglu_quantize_act, w4.w4a4_dequantize_act, w4.w4a4_rotate_quantize_act),
       "int8": (127, w4.w4a8_swiglu_quantize_act, w4.w4a8_dequantize_act, w4.w4a8_rotate_quantize_act)}


@pytest.mark.parametrize("fmt", list(FMT))
def test_scales_between_the_smallest_reciprocal_and_the_normal_range(fmt):
    dev = device()
    top, swiglu, back, plain = FMT[fmt]
    d = np.array([1.01, 1.5, 2.7, 3.9, 4.2, 9.0]) * 2.0 ** -128  # the last two are normal
    y = np.clip(np.random.default_rng(top).standard_normal((len(d), 32)) / 2, -0.99, 0.99) * (top * d)[:, None]
    y[:, 7] = top * d
    y[:, 11] = 0
    up = torch.from_numpy(y.astype(np.float32)).to(dev)
    gate = torch.ones_like(up)
    want = up.double().cpu().numpy() / (1 + np.exp(-1.0))
    # the scales of what silu(1) leaves: times 0.73; keep those whose reciprocal is finite
    scale = np.abs(want).max(axis=1) / top
    q = swiglu(gate, up, rotate=False)
    got = back(q).double().cpu().numpy()
    keep = scale > 1.001 * 2.0 ** -128
    assert keep.sum() >= 4 and (scale[keep] < 2.0 ** -126).sum() >= 2
    w, s = want[keep], scale[keep][:, None]
    u, tiny = 2.0 ** -24, 2.0 ** -150
    tol = 0.5 * s + np.abs(w) * (30 * u + 4 * u + 2 * u) + tiny * (top + 3)
    assert (np.abs(got[keep] - w) <= tol).all()
    assert (np.abs(got).max(axis=1)[keep] > 0).all() and not got[:, 11].any()
    # the plain quantiser reads the same rows back within the same bound
    v = torch.from_numpy(want.astype(np.float32)).to(dev)
    same = back(plain(v, rotate=False)).double().cpu().numpy()
    assert (np.abs(same[keep] - w) <= tol).all()
