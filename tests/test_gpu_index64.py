"""The quantisers', read-backs' and import's 64-bit index instances: operands of 2^32 elements and more from end to
end.  Rows 2^30 elements apart reach that with little work; the same rows close together go through the 32-bit
instances and have to give the same bits."""
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
M, K, LD = 5, 736, 1 << 30  # an odd number of blocks, a part of a scale tile
assert M * LD >= 1 << 32
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    return device()


def apart(dtype, dev, fill=None):
    t = torch.empty((M - 1) * LD + K + 64, dtype=dtype, device=dev).as_strided((M, K), (LD, 1))
    if fill is not None:
        t.copy_(fill)
    return t


def rows(seed, dtype, dev):
    return torch.randn(M, K, device=dev, generator=torch.Generator(dev).manual_seed(seed)).to(dtype)


def same(a, b):
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_to_mxfp4(dev, dtype):
    x = rows(1, dtype, dev)
    same(w4.mxfp4_rotate_quantize(apart(dtype, dev, x)), w4.mxfp4_rotate_quantize(x))


@pytest.mark.parametrize("call", [w4.w4a4_swiglu_quantize_act, w4.w4a8_swiglu_quantize_act, w4.mxfp4_swiglu_quantize])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu(dev, call, dtype):
    g, u = rows(2, dtype, dev), rows(3, dtype, dev)
    want = call(g, u)
    far = apart(dtype, dev, u)
    same(call(g, far), want)
    same(call(apart(dtype, dev, g), far), want)


@pytest.mark.parametrize("quantize,back", [(w4.w4a4_rotate_quantize_act, w4.w4a4_dequantize_act),
                                           (w4.w4a8_rotate_quantize_act, w4.w4a8_dequantize_act),
                                           (w4.mxfp4_rotate_quantize, w4.mxfp4_dequantize)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_read_back(dev, quantize, back, dtype):
    a = quantize(rows(4, F32, dev))
    y = apart(dtype, dev)
    y.fill_(7)
    y.as_strided((M, 64), (LD, 1), K).fill_(7)
    back(a, y=y)
    assert torch.equal(y, back(a, dtype=dtype)) and bool((y.as_strided((M, 64), (LD, 1), K) == 7).all())


@pytest.mark.parametrize("call", [w4.w4a4_rmsnorm_quantize_act, w4.w4a8_rmsnorm_quantize_act, w4.mxfp4_rmsnorm_quantize])
def test_norm(dev, call):
    x, r = rows(5, F32, dev), rows(6, BF16, dev)
    out = torch.empty_like(r)
    want = call(x, residual=r, residual_out=out)
    far = apart(BF16, dev)
    same(call(apart(F32, dev, x), residual=apart(BF16, dev, r), residual_out=far), want)
    assert torch.equal(far, out)


def test_import(dev):
    n, k = 131073, 32800  # 4.3e9 values
    assert n * k >= 1 << 32
    gen = torch.Generator(dev).manual_seed(7)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=dev, generator=gen)
    scales = torch.randint(0, 256, (n, k // 32), dtype=torch.uint8, device=dev, generator=gen)
    q = w4.mxfp4_import(codes, scales)
    assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales)
