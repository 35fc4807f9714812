"""Argument checks of the MXFP4 operators and of the fused quantisers.  Every call
fails validation, or has no rows, before anything is launched: no GPU is needed."""
import ctypes

import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from hadamard_rotated_w4a4_gb300 import _Act4Desc, _RmsNorm

FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return w4.load_library(build_if_missing=True)


def mx(rows=64, K=256, rotated=True, tag=None, codes=FAKE, scales=FAKE):
    return _Act4Desc(codes, scales, rows, K, tag if tag is not None else (w4.TAG_MXFP4 | (1 if rotated else 0)))


def status(lib, fn, *args):
    at = [ctypes.addressof(a) if isinstance(a, ctypes.Structure) else a for a in args]
    return w4.STATUS[getattr(lib, fn)(*at)]


def test_sizes(lib):
    assert lib.w4a4_mxfp4_codes_bytes(3, 96) == 144
    assert lib.w4a4_mxfp4_scales_bytes(1, 32) == 512
    assert lib.w4a4_mxfp4_scales_bytes(129, 160) == 2 * 2 * 512
    assert lib.w4a4_mxfp4_scales_bytes(4, 33) == 0


def test_gemm_refusals(lib):
    def call(w=mx(), a=mx(rows=8), y=FAKE, dt=1, ldy=64, ws=None, ws_bytes=0):
        return status(lib, "mxfp4_gemm", w, a, y, dt, ldy, ws, ws_bytes, None)

    assert call(w=mx(rotated=False)) == "W4A4_ERR_MISMATCH"
    assert call(w=mx(K=288)) == "W4A4_ERR_MISMATCH"
    assert call(w=mx(tag=w4.TAG_ACT4 | 1)) == "W4A4_ERR_INVALID_ARG"
    assert call(a=mx(tag=w4.TAG_Q4_0 | 1)) == "W4A4_ERR_INVALID_ARG"
    assert call(w=mx(K=48), a=mx(K=48)) == "W4A4_ERR_INVALID_ARG"
    assert call(w=mx(codes=None)) == "W4A4_ERR_INVALID_ARG"
    assert call(a=mx(scales=FAKE + 8)) == "W4A4_ERR_ALIGNMENT"
    assert call(y=None) == "W4A4_ERR_INVALID_ARG"
    assert call(y=FAKE + 2) == "W4A4_ERR_ALIGNMENT"
    assert call(y=FAKE + 1, dt=0) == "W4A4_ERR_ALIGNMENT"
    assert call(dt=2) == "W4A4_ERR_INVALID_ARG"
    assert call(ldy=63) == "W4A4_ERR_INVALID_ARG"
    assert call(w=mx(rows=65536 * 128), ldy=65536 * 128) == "W4A4_ERR_UNSUPPORTED"
    big, rows = mx(rows=20000, K=16384), mx(rows=1000, K=16384)  # 79 x 4 tiles: the last wave is cut
    need = lib.mxfp4_gemm_workspace_bytes(1000, 20000, 16384)
    assert need > 0 and need % 16 == 0
    assert call(w=big, a=rows, ldy=20000, ws=FAKE, ws_bytes=need - 16) == "W4A4_ERR_WORKSPACE"
    assert call(w=big, a=rows, ldy=20000, ws=FAKE + 8, ws_bytes=need) == "W4A4_ERR_ALIGNMENT"
    assert lib.mxfp4_gemm_workspace_bytes(1, 20000, 16384) == 0 and lib.mxfp4_gemm_workspace_bytes(1000, 20000, 33) == 0
    assert status(lib, "mxfp4_gemm", None, mx(), FAKE, 1, 64, None, 0, None) == "W4A4_ERR_INVALID_ARG"
    assert call(a=mx(rows=0), y=None) == "W4A4_OK"
    assert call(w=mx(rows=0), y=None, ldy=0) == "W4A4_OK"


def test_quantize_import_and_read_back_refusals(lib):
    d = mx()
    q = "mxfp4_rotate_quantize"
    assert status(lib, q, FAKE, 1, 4, 100, 100, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, FAKE, 1, 4, 64, 32, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, FAKE, 1, 4, 64, 66, 1, d, None) == "W4A4_ERR_ALIGNMENT"
    assert status(lib, q, FAKE, 0, 4, 64, 68, 1, d, None) == "W4A4_ERR_ALIGNMENT"
    assert status(lib, q, FAKE + 8, 1, 4, 64, 64, 1, d, None) == "W4A4_ERR_ALIGNMENT"
    assert status(lib, q, FAKE, 5, 4, 64, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, FAKE, 1, 4, 64, 64, 2, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, None, 1, 4, 64, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, FAKE, 1, 4, 64, 64, 1, None, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, FAKE, 1, -1, 64, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, q, FAKE, 1, 4, 64, 64, 1, mx(codes=None), None) == "W4A4_ERR_INVALID_ARG"
    e = mx(tag=0)
    assert status(lib, q, None, 1, 0, 64, 64, 1, e, None) == "W4A4_OK" and e.K == 64 and e.tag == w4.TAG_MXFP4 | 1
    i = "mxfp4_import"
    assert status(lib, i, FAKE + 4, FAKE, 4, 64, 1, d, None) == "W4A4_ERR_ALIGNMENT"
    assert status(lib, i, FAKE, None, 4, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, i, FAKE, FAKE, 4, 64, 3, d, None) == "W4A4_ERR_INVALID_ARG"
    for fn, good in (("mxfp4_dequantize", w4.TAG_MXFP4), ("w4a4_dequantize_act", w4.TAG_ACT4),
                     ("w4a8_dequantize_act", w4.TAG_ACT8)):
        assert status(lib, fn, mx(tag=w4.TAG_Q4_0), FAKE, 1, 256, None) == "W4A4_ERR_INVALID_ARG"
        assert status(lib, fn, mx(tag=good), FAKE, 1, 128, None) == "W4A4_ERR_INVALID_ARG"
        assert status(lib, fn, mx(tag=good), FAKE, 0, 260, None) == "W4A4_ERR_ALIGNMENT"
        assert status(lib, fn, mx(tag=good), None, 1, 256, None) == "W4A4_ERR_INVALID_ARG"
        assert status(lib, fn, mx(tag=good, rows=0), None, 1, 256, None) == "W4A4_OK"


NORMS = ("w4a4_rmsnorm_quantize_act", "w4a8_rmsnorm_quantize_act", "mxfp4_rmsnorm_quantize")


@pytest.mark.parametrize("fn", NORMS)
def test_norm_refusals(lib, fn):
    def call(out=None, **kw):
        n = _RmsNorm(**{**dict(x=FAKE, r=FAKE, r_out=FAKE, g=FAKE, M=4, K=64, ldx=64, ldr=64, ldr_out=64, x_dtype=1,
                               r_dtype=0, g_dtype=1, rotate=1, eps=1e-6), **kw})
        return status(lib, fn, n, out or _Act4Desc(FAKE, FAKE, 0, 0, 0), None)

    assert call(K=100) == "W4A4_ERR_INVALID_ARG"
    assert call(ldx=32) == "W4A4_ERR_INVALID_ARG"
    assert call(ldx=66) == "W4A4_ERR_ALIGNMENT"
    assert call(ldr=68) == "W4A4_ERR_ALIGNMENT"
    assert call(ldr_out=68) == "W4A4_ERR_ALIGNMENT"
    assert call(r_out=None) == "W4A4_ERR_INVALID_ARG"
    assert call(x=None) == "W4A4_ERR_INVALID_ARG"
    assert call(g=FAKE + 4) == "W4A4_ERR_ALIGNMENT"
    assert call(g_dtype=3) == "W4A4_ERR_INVALID_ARG"
    assert call(x_dtype=-1) == "W4A4_ERR_INVALID_ARG"
    assert call(rotate=2) == "W4A4_ERR_INVALID_ARG"
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == "W4A4_ERR_INVALID_ARG"
    assert call(K=65568, ldx=65568, ldr=65568, ldr_out=65568) == "W4A4_ERR_UNSUPPORTED"
    assert call(out=_Act4Desc(FAKE + 8, FAKE, 0, 0, 0)) == "W4A4_ERR_ALIGNMENT"
    assert call(M=0, x=None, r_out=None) == "W4A4_OK"
    assert status(lib, fn, None, _Act4Desc(FAKE, FAKE, 0, 0, 0), None) == "W4A4_ERR_INVALID_ARG"


@pytest.mark.parametrize("fn", ["w4a4_swiglu_quantize_act", "w4a8_swiglu_quantize_act", "mxfp4_swiglu_quantize"])
def test_swiglu_refusals(lib, fn):
    d = _Act4Desc(FAKE, FAKE, 0, 0, 0)
    assert status(lib, fn, FAKE, None, 1, 4, 64, 64, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, fn, None, FAKE, 1, 4, 64, 64, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, fn, FAKE, FAKE, 1, 4, 64, 64, 66, 1, d, None) == "W4A4_ERR_ALIGNMENT"
    assert status(lib, fn, FAKE, FAKE, 0, 4, 64, 63, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, fn, FAKE, FAKE, 7, 4, 64, 64, 64, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, fn, FAKE, FAKE, 1, 4, 65, 65, 65, 1, d, None) == "W4A4_ERR_INVALID_ARG"
    assert status(lib, fn, FAKE, FAKE, 1, 0, 64, 64, 64, 1, d, None) == "W4A4_OK"


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(2, 64)
    for call in (lambda: w4.mxfp4_rotate_quantize(x), lambda: w4.w4a8_rmsnorm_quantize_act(x),
                 lambda: w4.mxfp4_swiglu_quantize(x, x), lambda: w4.mxfp4_import(x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(w4.W4A4Error):
        w4.alloc_mxfp4(2, 48, "cpu")


def test_scale_view_undoes_the_tiles():
    q = w4.alloc_mxfp4(130, 160, "cpu")
    want = torch.arange(130 * 5, dtype=torch.int64).remainder(251).to(torch.uint8).view(130, 5)
    for r in range(130):
        for b in range(5):
            at = ((r // 128) * 2 + b // 4) * 512 + 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4
            q.scales_buf[at] = want[r, b]
    assert torch.equal(q.scales, want)
