"""Paths of the fused quantisers beside those of tests/test_gpu_fused_quant.py: loud gates, the scales' division,
int4 operands through the routed product."""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
import oracle
import test_gpu_fused_quant as fq
from w4a4_testutil import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


@pytest.mark.parametrize("fmt", list(fq.FMT))
def test_swiglu_of_loud_gates(dev, fmt, monkeypatch):
    """Gates up to 170.  The exponential is good to 2 + 1.18 |gate| units of 2 u, 406 u in all at 170, and the rest
    10 u; the rotation's magnitudes and roundings as derived there: (416 + 6) * 5.66 < 2560 = 8 * 320 u of the block's
    largest magnitude."""
    monkeypatch.setattr(fq, "U", 8 * fq.U)
    rng = np.random.default_rng(11)
    M, K = 67, 736
    gu = rng.standard_normal((M, 2 * K)) * 2
    gu[:, rng.integers(0, K, K // 50)] *= 20
    gu = torch.from_numpy(np.clip(gu, -170, 170).astype(np.float32)).to(dev)
    for dtype, rotate in ((fq.F32, True), (fq.BF16, False)):
        t = gu.to(dtype)
        g, u = (v.double().cpu().numpy() for v in (t[:, :K], t[:, K:]))
        assert np.abs(g).max() > 80
        fq.check_codes(fq.FMT[fmt][1](t[:, :K], t[:, K:], rotate=rotate), g / (1 + np.exp(-g)) * u, fmt, rotate)


@pytest.mark.parametrize("fmt,top", [("int4", 7), ("int8", 127)])
def test_scales_are_correctly_rounded_quotients(dev, fmt, top):
    """silu(64) is 64 in fp32, so a block of one value v has the scale fl(64 |v| / top): every mantissa at one
    exponent, a sample of them at the others."""
    v = (torch.arange(1 << 23, device=dev, dtype=torch.int64) + (127 << 23)).to(torch.int32).view(torch.float32)
    e = torch.randint(-120, 118, (1 << 20,), device=dev, generator=torch.Generator(dev).manual_seed(0))
    v = torch.cat((v, torch.ldexp(v[:: 8], e)))
    x = torch.zeros(v.numel(), 32, device=dev)
    x[:, 5] = v
    q = fq.FMT[fmt][1](torch.full((1, 1), 64.0, device=dev).expand(v.numel(), 32).contiguous(), x, rotate=False)
    want = (64 * v).double() / top  # 53 bits of the quotient, and no tie: top is odd
    assert torch.equal(q.scales[:, 0], want.float())


@pytest.mark.parametrize("aps", [False, True])
def test_int4_operands_through_the_routed_product(dev, aps):
    rng = np.random.default_rng(3)
    E, N, K, M, k = 8, 96, 256, 50, 2
    w = torch.from_numpy(rng.standard_normal((E * N, K)).astype(np.float32)).to(dev)
    wq = w4.h32_q4_0_pack_weights(w)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32)).to(dev)
    x = fq.data(5, M * k if aps else M, K, fq.F32, dev)
    codes = oracle.weight_codes_from_nibbles(oracle.unpack_nibbles(wq.codes.cpu().numpy())).astype(np.float64)
    W = (codes * np.repeat(wq.scales.double().cpu().numpy(), 32, axis=1)).reshape(E, N, K)
    for a in (w4.w4a4_rmsnorm_quantize_act(x), w4.w4a4_swiglu_quantize_act(x, x)):
        y = w4.w4a4_gemm_id(wq, E, a, ids, k, aps).double().cpu().numpy()
        A = w4.w4a4_dequantize_act(a).double().cpu().numpy()
        A = A.reshape(M, k, K) if aps else np.repeat(A[:, None], k, axis=1)
        sel = W[ids.cpu().numpy()]  # [M][k][N][K]
        R, mag = np.einsum("mknj,mkj->mkn", sel, A), np.einsum("mknj,mkj->mkn", np.abs(sel), np.abs(A))
        # block products exact; the fold: two products and an addition a block, each 2^-24 of the magnitudes; the
        # value read back is rounded once
        assert (np.abs(y - R) <= (3 * K / 32 + 1) * 2.0 ** -24 * mag).all()
