"""GPU parity of the fused norm and SwiGLU quantisers against 64 bits.

The fused kernels compute y in fp32 and then round it; the codes' rounding itself is
exact, so the read-back value must lie between the roundings of y - t and y + t, t
being the fp32 error of y, on the grid of the stored scale, and the scale must be
that of a block maximum within t.  t, in units u = 2^-24 of the block's largest
unrotated magnitude B:

* norm: h one rounding; a sum of K squares in at most 64 + 15 additions, halved by the
  root: 40; division, eps, rsqrt (2 ulp) and the two products: 8.  49 u.
* SwiGLU: the exponential is good to 2 + 1.18 |gate| units of 2u; |gate| < 8 here:
  12 * 2; sum, quotient (2 * 2) and product: 6.  30 u.
* rotation: 5 additions and a product on magnitudes of at most 32 B / sqrt 32 = 5.66 B:
  6 u each of those, and the error of y itself grows at most as much: (49 + 6) * 5.66 < 320.
t = 320 u B covers both, rotated or not.
"""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
import oracle
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FMT = {"int4": (w4.w4a4_rmsnorm_quantize_act, w4.w4a4_swiglu_quantize_act, w4.w4a4_dequantize_act),
       "int8": (w4.w4a8_rmsnorm_quantize_act, w4.w4a8_swiglu_quantize_act, w4.w4a8_dequantize_act),
       "mx": (w4.mxfp4_rmsnorm_quantize, w4.mxfp4_swiglu_quantize, w4.mxfp4_dequantize)}


@pytest.fixture(scope="module")
def dev():
    return device()


def rot64(y):
    return oracle.rotate_h32(y, dtype=np.float64)


def grid_round(v, fmt):
    if fmt == "mx":
        q = oracle.e2m1_code(v)
        return np.where(q >= 8, -1.0, 1.0) * oracle.E2M1[q & 7]
    top = 7 if fmt == "int4" else 127
    return np.clip(oracle.round_half_away(v), -top, top)


def check_codes(q, y, fmt, rotate):
    """q: quantised rows; y: their unrotated values in 64 bits."""
    M, K = y.shape
    B = np.abs(y).reshape(M, -1, 32).max(axis=-1)
    t = 320 * U * np.repeat(B, 32, axis=1)
    v = rot64(y) if rotate else y
    a = np.abs(v).reshape(M, -1, 32).max(axis=-1)
    if fmt == "mx":
        s = np.exp2(q.scales.cpu().numpy().astype(np.float64) - 127)
        # floor(log2) of a maximum within t: the scale is that of a - t or of a + t
        lo, hi = (np.exp2(np.floor(np.log2(np.maximum(a + k * t[:, ::32], 2.0 ** -125))) - 2) for k in (-1, 1))
        assert ((s == lo) | (s == hi) | (a == 0)).all()
    else:
        s = q.scales.cpu().numpy().astype(np.float64)
        # the stored scale: the maximum's error and one division
        assert (np.abs(s * (7 if fmt == "int4" else 127) - a) <= t[:, ::32] + 2 * U * a).all()
    S = np.repeat(s, 32, axis=1)
    back = FMT[fmt][2](q).double().cpu().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        # two fp32 roundings of y / s, 4 u of it, beside t
        w = np.where(S > 0, v / S, 0.0)
        e = np.where(S > 0, t / S, 0.0) + 4 * U * np.abs(w)
    lo, hi = grid_round(w - e, fmt) * S, grid_round(w + e, fmt) * S
    slack = 2 * U * np.abs(back)  # code * scale rounds once
    assert (back >= lo - slack).all() and (back <= hi + slack).all()


def data(seed, M, K, dtype, dev, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32) * np.float32(scale)
    x[:, rng.integers(0, K, max(1, K // 100))] *= 20
    return torch.from_numpy(x).to(dev).to(dtype)


def norm64(h, g, eps):
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return y if g is None else y * g.double().cpu().numpy()


F32, BF16 = torch.float32, torch.bfloat16
# K of one block, below and above a warp's row, odd block counts, several chunks a thread
NORM_SHAPES = [(1, 32), (1, 5120), (3, 64), (70, 96), (33, 224), (5, 256), (9, 288), (200, 736), (700, 8224), (2, 17408),
               (4, 33024), (1, 65536)]
# many rows
NORM_SHAPES += [(457, 288), (500, 5120), (3000, 416), (1000, 9216)]


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm(dev, M, K, fmt):
    rng = np.random.default_rng(M + K)
    for dx, dr, dg, rotate in ((F32, BF16, F32, True), (BF16, F32, BF16, False), (BF16, BF16, F32, True),
                               (F32, None, None, True)):
        x = data(K, M, K, dx, dev)
        r = None if dr is None else data(K + 1, M, K, dr, dev, 2.0)
        g = None if dg is None else torch.from_numpy((1 + 0.1 * rng.standard_normal(K)).astype(np.float32)).to(dev).to(dg)
        h = x.double() + (0 if r is None else r.double())
        if r is None:
            q = FMT[fmt][0](x, g, eps=1e-6, rotate=rotate)
        else:
            out, keep = torch.empty_like(r), r.clone()
            q = FMT[fmt][0](x, g, eps=1e-6, residual=r, residual_out=out, rotate=rotate)
            assert torch.equal(r, keep)
            # one fp32 rounding, then one to r's type
            assert torch.equal(out, (x.float() + r.float()).to(dr))
        check_codes(q, norm64(h.cpu().numpy(), g, 1e-6), fmt, rotate)


@pytest.mark.parametrize("M", [50, 1500])
@pytest.mark.parametrize("dr", [F32, BF16])
def test_norm_in_place_strided_and_expanded(dev, dr, M):
    K = 416
    x, r = data(1, M, K, F32, dev), data(2, M, K, dr, dev)
    want_r = (x + r.float()).to(dr)
    wide = torch.full((M, K + 32), 7.0, dtype=dr, device=dev)
    wide[:, :K] = r
    xw = torch.full((M, K + 64), float("nan"), device=dev)
    xw[:, 32:K + 32] = x
    q = w4.w4a4_rmsnorm_quantize_act(xw[:, 32:K + 32], residual=wide[:, :K])
    assert torch.equal(wide[:, :K], want_r) and bool((wide[:, K:] == 7).all())
    check_codes(q, norm64((x.double() + r.double()).cpu().numpy(), None, 1e-6), "int4", True)
    # the expanded operand holds the same codes: a + 8
    nib = oracle.act_codes_from_nibbles(oracle.unpack_nibbles(q.codes.cpu().numpy()))
    assert np.array_equal(q.expanded[: M * K].view(M, K).cpu().numpy().astype(np.int64), nib + 8)


@pytest.mark.parametrize("fmt", list(FMT))
def test_norm_special_rows(dev, fmt):
    K = 256
    x = data(4, 6, K, F32, dev)
    x[1] = 0
    x[2, 40] = float("nan")
    x[3, 40] = float("inf")
    x[4] = 1e25  # the squares overflow: the norm is infinite, y is 0
    norm, _, back = FMT[fmt]
    v = back(norm(x, eps=1e-6, rotate=False)).cpu()
    alone = back(norm(x[:1].contiguous(), eps=1e-6, rotate=False)).cpu()
    assert torch.equal(v[0], alone[0])
    assert not bool(v[1].any()) and bool(torch.isnan(v[2]).all()) and not bool(v[4].any())
    bad = torch.zeros(K, dtype=torch.bool)
    bad[32:64] = True
    assert torch.equal(torch.isnan(v[3]), bad) and not bool(v[3][~bad].any())
    assert bool(torch.isnan(back(norm(x[1:2].contiguous(), eps=0.0, rotate=False))).all())


@pytest.mark.parametrize("fmt", list(FMT))
def test_tiny_blocks(dev, fmt):
    """Blocks down to the smallest fp32 values: finite, zeros stay zeros, and MXFP4 keeps what fits 2^-127 scales."""
    one = torch.ones(1, 160, device=dev)
    # silu(1) is a constant c: gate = 1 passes up * c through to the codes
    up = torch.zeros(1, 160, device=dev)
    up[0, 0], up[0, 33], up[0, 64], up[0, 97], up[0, 128] = 1e-30, 1e-36, 1e-38, 1e-44, 1.0
    v = FMT[fmt][2](FMT[fmt][1](one, up, rotate=False)).cpu()[0]
    at = torch.zeros(160, dtype=torch.bool)
    at[[0, 33, 64, 97, 128]] = True
    assert bool(torch.isfinite(v).all()) and not bool(v[~at].any())
    c = 1 / (1 + np.exp(-1.0))
    for k, x in ((0, 1e-30), (128, 1.0)):
        assert abs(float(v[k]) - c * x) <= (0.25 if fmt == "mx" else 1e-6) * c * x
    assert 0 <= float(v[33]) <= 1.3e-36 and 0 <= float(v[64]) <= 1.3e-38


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("M,K", [(1, 32), (1, 17408), (67, 768), (33, 736), (300, 96)])
def test_swiglu(dev, M, K, fmt):
    rng = np.random.default_rng(K)
    for dtype, rotate in ((F32, True), (BF16, True), (F32, False)):
        gu = torch.from_numpy(np.clip(rng.standard_normal((M, 2 * K)) * 2, -7.9, 7.9).astype(np.float32)).to(dev).to(dtype)
        gate, up = gu[:, :K], gu[:, K:]  # the halves of one product's output
        q = FMT[fmt][1](gate, up, rotate=rotate)
        g, u = gate.double().cpu().numpy(), up.double().cpu().numpy()
        check_codes(q, g / (1 + np.exp(-g)) * u, fmt, rotate)
        same = FMT[fmt][1](gate.contiguous(), up.contiguous(), rotate=rotate)
        assert torch.equal(q.codes, same.codes) and torch.equal(q.scales, same.scales)


@pytest.mark.parametrize("fmt", list(FMT))
def test_swiglu_special_values(dev, fmt):
    gate, up = torch.ones(1, 256, device=dev), torch.ones(1, 256, device=dev)
    gate[0, 0:32], gate[0, 32:64] = 200.0, -200.0  # 200 and, to fp32, 0
    gate[0, 70] = float("nan")
    up[0, 100] = float("inf")
    gate[0, 130], up[0, 130] = -200.0, 3.0
    v = FMT[fmt][2](FMT[fmt][1](gate, up, rotate=False)).cpu()[0]
    assert torch.isnan(v[64:128]).all() and not torch.isnan(v[:64]).any() and not torch.isnan(v[128:]).any()
    assert not v[32:64].any() and v[130] == 0
    assert torch.allclose(v[:32], torch.full((32,), 200.0), rtol=0.05)


def test_norm_feeds_the_products(dev):
    """The fused operands are what the package's products take: the same codes, the same result."""
    import synth_inputs as si
    d = si.random_dense(40, 512, 96, seed=3)
    w = torch.from_numpy(d["w"]).to(dev)
    x = data(7, 40, 512, F32, dev)
    y64 = norm64(x.double().cpu().numpy(), None, 1e-6)
    y = torch.from_numpy(y64.astype(np.float32)).to(dev)
    wq = w4.h32_q4_0_pack_weights(w)
    pairs = [(w4.w4a4_gemm(wq, w4.w4a4_rmsnorm_quantize_act(x)), w4.w4a4_gemm(wq, w4.w4a4_rotate_quantize_act(y))),
             (w4.w4a8_gemm(wq, w4.w4a8_rmsnorm_quantize_act(x)), w4.w4a8_gemm(wq, w4.w4a8_rotate_quantize_act(y))),
             (w4.mxfp4_gemm(w4.mxfp4_rotate_quantize(w), w4.mxfp4_rmsnorm_quantize(x)),
              w4.mxfp4_gemm(w4.mxfp4_rotate_quantize(w), w4.mxfp4_rotate_quantize(y)))]
    for a, b in pairs:  # a code may move by a step where y sits on a boundary: a hundredth of the result covers it
        assert float((a - b).norm()) <= 0.01 * float(b.norm())


def test_fused_on_another_stream(dev):
    x, r = data(1, 64, 1024, BF16, dev), data(2, 64, 1024, BF16, dev)
    want, other = w4.w4a8_rmsnorm_quantize_act(x, residual=r.clone()), r.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = w4.w4a8_rmsnorm_quantize_act(x, residual=other, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
