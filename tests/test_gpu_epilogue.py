"""The MXFP4 product with bias, activation and residual against 64 bits.

The product's sums are those of mxfp4_gemm, whose result stands in for them: what is tested is
act(p + bias) + residual.  fp32: p + bias rounds once, U |x|.  SiLU and tanh-GELU: z = x (c1 + c3 x^2) 4 U |z|, and the
exponential 2 + 1.18 |z| units of 2 U; with the sum and the quotient (3 ulp) y is off by (6 |z| + 14) U |y| at most, and
d act / dx (at most 1.2) times U |x|.  GELU: erf 2 ulp of a value of at most 1, 1 + erf one, two products: 8 U |x|.  The
residual's sum: U |y|.  Taken together: (6 |z| + 20) U (|x| + |residual|), |z| up to 30 where y is not negligible (beyond,
exp(-z) has no bit in 1 + exp(-z), or y is under 1e-12 |x|).
"""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return device()


def act_64(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x / 2 ** 0.5)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3))
    return x


def operands(seed, M, N, K, dev, scale=1.0):
    gen = torch.Generator(dev).manual_seed(seed)
    w = w4.mxfp4_rotate_quantize(torch.randn(N, K, device=dev, generator=gen) * K ** -0.5 * scale)
    return w, w4.mxfp4_rotate_quantize(torch.randn(M, K, device=dev, generator=gen)), gen


def check(y, p, bias, act, residual):
    x = p.double() if bias is None else p.double() + bias.double()
    want = act_64(x, act)
    size = x.abs() + want.abs()
    if residual is not None:
        want = want + residual.double()
        size = size + residual.double().abs()
    tol = (6 * x.abs().mul(1.6).clamp(max=30) + 20) * U * size + 1e-12 * x.abs()
    tol = tol + (torch.finfo(y.dtype).eps / 2) * (want.abs() + tol)
    off = (y.double() - want).abs()
    assert (off <= tol).all(), f"off by {float((off - tol).max()):.3e} past {float(tol.max()):.3e}"


SHAPES = [(1, 128, 64), (1, 7168, 5120), (3, 200, 96), (17, 129, 736), (64, 5120, 5120), (77, 1000, 736), (128, 2048, 2048),
          (200, 20000, 320), (333, 4600, 1184), (257, 20001, 160), (1024, 5120, 17408)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_epilogue(dev, M, N, K, dtype):
    w, a, gen = operands(M + N, M, N, K, dev)
    p = w4.mxfp4_gemm(w, a)
    bias = torch.randn(N, device=dev, generator=gen)
    res = torch.randn(M, N, device=dev, generator=gen)
    for act in (None, "relu", "silu", "gelu", "gelu_tanh"):
        check(w4.mxfp4_gemm_epilogue(w, a, bias, act, res, dtype=dtype), p, bias, act, res)
    check(w4.mxfp4_gemm_epilogue(w, a, None, "gelu", None, dtype=dtype), p, None, "gelu", None)
    rb = res.to(torch.bfloat16)
    check(w4.mxfp4_gemm_epilogue(w, a, None, None, rb, dtype=dtype), p, None, None, rb)
    check(w4.mxfp4_gemm_epilogue(w, a, bias, "none", rb, dtype=dtype, ws=None), p, bias, None, rb)
    plain = w4.mxfp4_gemm_epilogue(w, a, dtype=dtype)
    assert torch.equal(plain, w4.mxfp4_gemm(w, a, dtype=dtype))  # nothing asked for: the product itself
    w4.w4a4_check()


def test_epilogue_of_loud_sums(dev):
    """Sums in the hundreds, where exponentials overflow and vanish."""
    w, a, gen = operands(5, 40, 300, 512, dev, scale=100.0)
    p = w4.mxfp4_gemm(w, a)
    assert p.abs().max() > 200
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        y = w4.mxfp4_gemm_epilogue(w, a, None, act)
        assert torch.isfinite(y).all()
        check(y, p, None, act, None)


@pytest.mark.parametrize("M,N", [(5, 300), (300, 20002)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_epilogue_in_place_and_strided(dev, M, N, dtype):
    """y += W a on the residual itself, in a wider buffer whose other columns stay."""
    w, a, gen = operands(6, M, N, 288, dev)
    p = w4.mxfp4_gemm(w, a)
    buf = torch.randn(M, N + 11, device=dev, generator=gen).to(dtype)
    was = buf.clone()
    y = buf[:, 3:3 + N]
    assert w4.mxfp4_gemm_epilogue(w, a, residual=y, y=y) is y
    check(y, p, None, None, was[:, 3:3 + N])
    assert torch.equal(buf[:, :3], was[:, :3]) and torch.equal(buf[:, 3 + N:], was[:, 3 + N:])
    other = was[:, 8:8 + N]  # another stride than y's
    check(w4.mxfp4_gemm_epilogue(w, a, residual=other, dtype=dtype), p, None, None, other)


def test_epilogue_reads_what_the_call_before_wrote(dev):
    """The residual and the bias of one product are the output of the one in front of it on the stream."""
    for M in (1, 40, 400):
        w, a, gen = operands(7, M, 5120, 160, dev)
        y0 = w4.mxfp4_gemm(w, a)
        for _ in range(20):
            y = w4.mxfp4_gemm(w, a)
            y = w4.mxfp4_gemm_epilogue(w, a, residual=y, y=y)
            y = w4.mxfp4_gemm_epilogue(w, a, bias=y[0], residual=y)
        want = (y0.double() * 2 + y0.double() + 2 * y0[:1].double())
        assert (y.double() - want).abs().max() <= 8 * U * want.abs().max()


@pytest.mark.parametrize("M", [3, 300])
def test_epilogue_of_infinities(dev, M):
    """What a bias of infinity or NaN makes: its column alone, and there what the formula gives."""
    w, a, gen = operands(5, M, 200, 96, dev)
    bias = torch.zeros(200, device=dev)
    bias[7], bias[8], bias[130] = float("inf"), float("nan"), -float("inf")
    p = w4.mxfp4_gemm(w, a)
    for act in (None, "relu", "silu", "gelu", "gelu_tanh"):
        y = w4.mxfp4_gemm_epilogue(w, a, bias, act)
        assert (y[:, 7] == float("inf")).all() and torch.isnan(y[:, 8]).all()
        if act in (None, "relu"):
            assert (y[:, 130] == (0.0 if act else -float("inf"))).all()
        rest = bias == 0
        check(y[:, rest], p[:, rest], None, act, None)


def test_epilogue_refusals(dev):
    w, a, gen = operands(8, 4, 96, 64, dev)
    z = lambda *s, **k: torch.zeros(*s, device=dev, **k)  # noqa: E731
    for kw in (dict(bias=z(95)), dict(bias=z(96, dtype=torch.bfloat16)), dict(bias=z(192)[::2]), dict(bias=torch.zeros(96)),
               dict(activation="tanh"), dict(residual=z(4, 95)), dict(residual=z(4, 96, dtype=torch.float16)), dict(y=z(4, 97)),
               dict(residual=torch.zeros(4, 96))):
        with pytest.raises(ValueError):
            w4.mxfp4_gemm_epilogue(w, a, **kw)
    with pytest.raises(w4.W4A4Error):
        w4.mxfp4_gemm_epilogue(w, a, dtype=torch.float16)
    with pytest.raises(w4.W4A4Error):  # the residual's storage as y, of another type
        r = z(4, 96)
        w4.mxfp4_gemm_epilogue(w, a, residual=r, y=r.view(torch.bfloat16)[:, :96])
