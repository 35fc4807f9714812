"""The MXFP4 product's epilogue within the error of each of its steps, U = 2^-24 a rounding to fp32.

Without an activation, and with ReLU, the steps are sum + bias, max and + residual: each rounded once, so the result is
that of the same steps in fp32, bit for bit.

x = p + bias is the activation's input, off by U |x| where there is a bias; no activation has a slope above 1.13.
SiLU, and GELU by tanh: y = x / (1 + e), e = exp(-z) = 2^u.  u is off by 2 U of itself (SiLU: the constant, the product) or by
6 U (tanh: a constant's three roundings, x^2, a fused multiply-add, the product), so e by that of |z| and by the exponential's
4 U; 1 + e by e / (1 + e) of e's and U; the reciprocal 2 U, the product U.  Where e or the reciprocal leaves fp32's range, y is
under 1e-35.
GELU: y = max(x, 0) - |x| q, q = erfc(|x| / sqrt 2) / 2 as t (c1 + t (c2 + ..)) E, E = exp(-x^2 / 2), off by 0.75e-7 as the
formula says.  t = 1 / (1 + c |x|) is off by 3 U of the constant, U of the sum and the reciprocal's 2 U, and t dq/dt is at
most 8.1 E (the sum of i |ci|): 49 U.  Horner's five steps round sums of at most 2.24, their constants once: 14 U.  E is off
by 3 U x^2 / 2 and the exponential's 4 U, beside a t (c1 + ..) of at most 1 / 2, and its product by U, then the last fused
multiply-add by U |y|.
"""
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

# one token, a few, a split of K over CTAs, one wave of pairs, tiles cut over pairs, ragged either way
SHAPES = [(1, 7168, 5120), (3, 200, 96), (17, 129, 736), (64, 5120, 5120), (333, 4600, 1184), (257, 2001, 160), (700, 5000, 4000)]


@pytest.fixture(scope="module")
def dev():
    return device()


def operands(seed, M, N, K, dev, size):
    gen = torch.Generator(dev).manual_seed(seed)
    w = w4.mxfp4_rotate_quantize(torch.randn(N, K, device=dev, generator=gen) * K ** -0.5 * size)
    a = w4.mxfp4_rotate_quantize(torch.randn(M, K, device=dev, generator=gen))
    bias = torch.randn(N, device=dev, generator=gen) * size
    return w, a, bias, torch.randn(M, N, device=dev, generator=gen) * size


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bias_relu_and_residual_are_fp32s_own_steps(dev, M, N, K):
    w, a, bias, res = operands(M, M, N, K, dev, 1.0)
    p = w4.mxfp4_gemm(w, a)
    for dtype in (torch.float32, torch.bfloat16):
        for act in (None, "relu"):
            for b in (None, bias):
                for r in (None, res, res.to(torch.bfloat16)):
                    want = p if b is None else p + b
                    want = want if act is None else torch.relu(want)
                    want = (want if r is None else want + r.float()).to(dtype)
                    got = w4.mxfp4_gemm_epilogue(w, a, b, act, r, dtype=dtype)
                    assert torch.equal(got, want), (dtype, act, b is None, r is None)


def activation(x, act):
    """Its value in 64 bits, and what the kernel's fp32 may be off by for this x."""
    a = x.abs()
    if act == "gelu":
        E = torch.exp(-x * x / 2)
        y = 0.5 * x * torch.erfc(-x / 2 ** 0.5)
        return y, 0.75e-7 * a + U * a * E * (49 + 14 + (1.5 * x * x + 5) / 2) + U * y.abs()
    z, n = (x, 2) if act == "silu" else (2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3), 6)
    y = x * torch.sigmoid(z)
    return y, U * y.abs() * ((n * z.abs() + 4) * torch.sigmoid(-z) + 4) + 1e-35


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("size", [0.1, 1.0, 30.0])
def test_activations_within_their_steps(dev, M, N, K, act, size):
    w, a, bias, res = operands(M + 1, M, N, K, dev, size)
    p = w4.mxfp4_gemm(w, a).double()
    for b in (None, bias):
        x = p if b is None else p + b.double()
        y, off = activation(x, act)
        if b is not None:
            off = off + 1.13 * U * x.abs()
        for r in (None, res):
            want = y if r is None else y + r.double()
            tol = off if r is None else off + U * (want.abs() + off)
            got = w4.mxfp4_gemm_epilogue(w, a, b, act, r).double()
            worst = ((got - want).abs() - tol).max()
            assert worst <= 0, f"off by {float(worst):.2e} past {float(tol.max()):.2e}"
            got = w4.mxfp4_gemm_epilogue(w, a, b, act, r, dtype=torch.bfloat16).double()
            assert ((got - want).abs() <= tol + torch.finfo(torch.bfloat16).eps / 2 * (want.abs() + tol)).all()
