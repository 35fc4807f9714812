"""GPU parity of the MXFP4 quantiser, import, reading back and product.

Codes and scale bytes match the oracle bit for bit.  Products: the operands' values
are exact, so an output's error is that of the fp32 sums alone, at most 2^-23 of the
sum of magnitudes per addition (rounded or truncated), K additions: K 2^-23 (|a| |w|^T).
A bf16 output is the fp32 output rounded to nearest even, bit for bit.
"""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
import oracle
from w4a4_testutil import bf16_tensor, device, f32_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def rows(seed, M, K):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 100))] *= 20
    return x


def same_codes(q, ref):
    assert np.array_equal(q.codes.cpu().numpy(), ref["codes"])
    assert np.array_equal(q.scales.cpu().numpy(), ref["scales"])


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 5120), (3, 96), (5, 160), (129, 1024), (33, 736), (300, 2080)])
def test_quantiser_bit_exact(dev, M, K, rotate):
    x = rows(M + K, M, K)
    q = w4.mxfp4_rotate_quantize(f32_tensor(x, dev), rotate=rotate)
    assert q.rotated == rotate
    same_codes(q, oracle.quantize_mxfp4(x, rotate=rotate))
    bits = oracle.round_bf16(x)
    same_codes(w4.mxfp4_rotate_quantize(bf16_tensor(bits, dev), rotate=rotate),
               oracle.quantize_mxfp4(oracle.bf16_to_f32(bits), rotate=rotate))


def special_blocks():
    x = np.zeros((1, 32 * 12), np.float32)
    b = x.reshape(12, 32)
    b[0, :14] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -2.5, -5, 7.99, -7.99]
    b[2, 3] = np.nan
    b[3, 31] = np.inf
    b[4, 8] = -np.inf
    b[5, 0], b[5, 1] = 2.0 ** -126, 2.0 ** -149
    b[6, 30] = 2.0 ** -149
    b[7, 5], b[7, 6] = 3.4028235e38, -1e38
    b[8, :] = -0.0
    b[9, 17], b[9, 16] = 2.0 ** -125, 2.0 ** -128
    b[10, :] = np.arange(32) / 4 - 4
    b[11, 7] = np.nextafter(np.float32(8), np.float32(0))
    return x


def test_quantiser_special_blocks(dev):
    x = special_blocks()
    ref = oracle.quantize_mxfp4(x, rotate=False)
    q = w4.mxfp4_rotate_quantize(f32_tensor(x, dev), rotate=False)
    same_codes(q, ref)
    back = w4.mxfp4_dequantize(q).cpu().numpy()
    # 2^-127 times a code is below fp32's normal range but exact
    assert np.array_equal(back.astype(np.float64), oracle.mxfp4_values(ref["codes"], ref["scales"]), equal_nan=True)


def test_nan_stays_in_its_block_when_rotated(dev):
    x = rows(3, 4, 128)
    x[1, 40], x[2, 127] = np.nan, np.inf
    got = w4.mxfp4_dequantize(w4.mxfp4_rotate_quantize(f32_tensor(x, dev))).cpu().numpy()
    want = np.zeros((4, 128), bool)
    want[1, 32:64] = want[2, 96:] = True
    assert np.array_equal(np.isnan(got), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_and_reading_back(dev, dtype):
    x = torch.from_numpy(rows(9, 37, 224)).to(dev).to(dtype)
    big = torch.full((37, 224 + 48), float("nan"), dtype=dtype, device=dev)
    big[:, 16:240] = x
    a, b = w4.mxfp4_rotate_quantize(x), w4.mxfp4_rotate_quantize(big[:, 16:240])
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    want = oracle.mxfp4_values(a.codes.cpu().numpy(), a.scales.cpu().numpy())
    for out in (torch.float32, torch.bfloat16):  # every value fits both types
        y = torch.full((37, 224 + 16), 7.0, dtype=out, device=dev)
        w4.mxfp4_dequantize(a, y=y[:, :224])
        assert np.array_equal(y[:, :224].double().cpu().numpy(), want) and bool((y[:, 224:] == 7).all())


@pytest.mark.parametrize("M,K", [(1, 32), (5, 160), (300, 736)])
def test_import_is_bit_exact(dev, M, K):
    rng = np.random.default_rng(K)
    codes = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
    scales = rng.integers(0, 256, (M, K // 32), dtype=np.uint8)
    q = w4.mxfp4_import(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev))
    same_codes(q, {"codes": codes, "scales": scales})
    if K % 128:  # the last tile's unused blocks hold a finite scale
        tiles = q.scales_buf.view(-1, (K + 127) // 128, 32, 4, 4)[:, -1].permute(0, 2, 1, 3).reshape(-1, 4)[:M]
        assert not bool(tiles[:, K // 32 % 4:].any())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,K", [(1, 32), (7, 96), (130, 736)])
def test_int_formats_read_back(dev, bits, M, K):
    x = f32_tensor(rows(M, M, K), dev)
    if bits == 4:
        a = w4.w4a4_rotate_quantize_act(x)
        q = oracle.act_codes_from_nibbles(oracle.unpack_nibbles(a.codes.cpu().numpy()))
        back = w4.w4a4_dequantize_act
    else:
        a = w4.w4a8_rotate_quantize_act(x)
        q = a.codes.cpu().numpy().astype(np.int64)
        back = w4.w4a8_dequantize_act
    want = (q.astype(np.float32) * np.repeat(a.scales.cpu().numpy(), 32, axis=1)).astype(np.float32)
    assert np.array_equal(back(a).cpu().numpy(), want)
    assert torch.equal(back(a, dtype=torch.bfloat16).cpu(), torch.from_numpy(want).to(torch.bfloat16))


# ----------------------------------------------------------------- the product
def operands(dev, M, K, N, seed=0, rotate=True):
    w = rows(seed + 1, N, K) * np.float32(0.02)
    x = rows(seed + 2, M, K)
    qw = w4.mxfp4_rotate_quantize(f32_tensor(w, dev), rotate=rotate)
    qa = w4.mxfp4_rotate_quantize(f32_tensor(x, dev), rotate=rotate)
    return qw, qa


def values(q):
    return oracle.mxfp4_values(q.codes.cpu().numpy(), q.scales.cpu().numpy())


def check_product(qw, qa, y):
    W, A = values(qw), values(qa)
    R = (A @ W.T).astype(np.float32)  # what is below fp32's range is 0
    tol = qw.K * 2.0 ** -23 * (np.abs(A) @ np.abs(W).T)
    assert (np.abs(y.double().cpu().numpy() - R) <= tol).all()


# M around each token tile, K with an odd number of blocks, of scale tiles and of
# stages, N around the weight tile
SHAPES = [(1, 32, 1), (1, 5120, 640), (2, 64, 127), (8, 2048, 128), (15, 96, 129), (16, 736, 130), (17, 128, 256),
          (32, 160, 33), (33, 5120, 260), (64, 256, 100), (65, 288, 384), (127, 1056, 40), (128, 512, 128),
          (129, 2080, 513), (255, 64, 257), (256, 320, 128), (257, 96, 1000), (300, 2048, 640), (513, 736, 129),
          (700, 17408, 136)]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(dev, M, K, N, out):
    qw, qa = operands(dev, M, K, N, seed=M + K + N)
    # a canary around a strided output: nothing but [M][N] is written
    y = torch.full((M + 2, N + 8), 7.0, dtype=out, device=dev)
    w4.mxfp4_gemm(qw, qa, y=y[1:M + 1, :N])
    w4.w4a4_check()
    got = y[1:M + 1, :N]
    if out == torch.float32:
        check_product(qw, qa, got)
    else:
        assert torch.equal(got, w4.mxfp4_gemm(qw, qa).to(out))
    assert bool((y[0] == 7).all()) and bool((y[-1] == 7).all()) and bool((y[:, N:] == 7).all())


# more tiles than CTA pairs (76 on a GB300), the last wave mostly empty: its stages are
# cut over the pairs; with whole waves in front of it and without, ragged in M, N and K
@pytest.mark.parametrize("M,K,N", [(200, 7456, 19500), (300, 7456, 29200), (257, 8224, 10100)])
def test_product_with_the_last_wave_cut(dev, M, K, N):
    assert w4.mxfp4_gemm_workspace_bytes(M, N, K) > 0
    gen = torch.Generator("cuda").manual_seed(M)
    w, x = (torch.randn(r, K, device=dev, generator=gen) for r in (N, M))
    qw, qa = w4.mxfp4_rotate_quantize(w * 0.02), w4.mxfp4_rotate_quantize(x)
    W, A = w4.mxfp4_dequantize(qw).double(), w4.mxfp4_dequantize(qa).double()
    R, tol = A @ W.T, K * 2.0 ** -23 * (A.abs() @ W.abs().T)
    y = w4.mxfp4_gemm(qw, qa)
    assert bool(((y.double() - R).abs() <= tol).all())
    assert bool(((w4.mxfp4_gemm(qw, qa, ws=False).double() - R).abs() <= tol).all())
    for _ in range(3):  # the workspace is left as it was found, and the sums' order is fixed
        assert torch.equal(w4.mxfp4_gemm(qw, qa), y)
    assert torch.equal(w4.mxfp4_gemm(qw, qa, dtype=torch.bfloat16), y.to(torch.bfloat16))
    w4.w4a4_check()


def test_workspace_shared_with_the_int4_product(dev):
    """One workspace serves both products of a stream, in any order, whatever each leaves in it."""
    M, K, N = 257, 8224, 10100
    qw, qa = operands(dev, M, K, N)
    x, w = f32_tensor(rows(2, 300, 1024), dev), f32_tensor(rows(1, 640, 1024) * np.float32(0.02), dev)
    wq, aq = w4.h32_q4_0_pack_weights(w), w4.w4a4_rotate_quantize_act(x)
    need = max(w4.mxfp4_gemm_workspace_bytes(M, N, K), w4.w4a4_gemm_workspace_bytes(300, 640, 1024))
    assert w4.mxfp4_gemm_workspace_bytes(M, N, K) > 0 and w4.w4a4_gemm_workspace_bytes(300, 640, 1024) > 0
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    want = w4.mxfp4_gemm(qw, qa, ws=ws), w4.w4a4_gemm(wq, aq, ws=torch.zeros(need, dtype=torch.uint8, device=dev))
    assert not bool(ws[: 1 << 20].any())  # the counters' part is left as it was found
    for _ in range(3):
        assert torch.equal(w4.w4a4_gemm(wq, aq, ws=ws), want[1])
        assert torch.equal(w4.mxfp4_gemm(qw, qa, ws=ws), want[0])
    assert not bool(ws[: 1 << 20].any())
    w4.w4a4_check()


def test_product_does_not_depend_on_what_ran_before(dev):
    qw, qa = operands(dev, 200, 1056, 300)
    y = w4.mxfp4_gemm(qw, qa)
    for M, K, N in ((1, 4096, 256), (600, 512, 512), (31, 96, 77)):
        w4.mxfp4_gemm(*operands(dev, M, K, N))
        assert torch.equal(w4.mxfp4_gemm(qw, qa), y)


def test_rows_of_a_batch_are_the_single_rows(dev):
    """A token's result is the same sum whatever tile it sits in, up to the fp32 sums' order."""
    qw, qa = operands(dev, 40, 800, 200)
    y = w4.mxfp4_gemm(qw, qa)
    x = f32_tensor(rows(2, 40, 800), dev)
    for m in (0, 17, 39):
        one = w4.mxfp4_rotate_quantize(x[m:m + 1])
        check_product(qw, one, w4.mxfp4_gemm(qw, one))
        assert torch.allclose(w4.mxfp4_gemm(qw, one)[0], y[m], rtol=0, atol=float(y.abs().max()) * 800 * 2.0 ** -23)


def test_zero_and_extreme_scales(dev):
    rng = np.random.default_rng(5)
    M, K, N = 20, 320, 140
    wc, ac = (rng.integers(0, 256, (r, K // 2), dtype=np.uint8) for r in (N, M))
    ws = rng.integers(100, 150, (N, K // 32), dtype=np.uint8)
    asc = rng.integers(100, 150, (M, K // 32), dtype=np.uint8)
    ws[3], asc[4], wc[5] = 0, 0, 0  # 2^-127 scales, a row of zero codes
    t = lambda v: torch.from_numpy(v).to(dev)  # noqa: E731
    qw, qa = w4.mxfp4_import(t(wc), t(ws)), w4.mxfp4_import(t(ac), t(asc))
    y = w4.mxfp4_gemm(qw, qa)
    check_product(qw, qa, y)
    assert not bool(y[:, 5].any())


def test_nan_scale_reaches_its_row_only(dev):
    w, x = rows(1, 150, 192), rows(2, 70, 192)
    w[9, 100], x[66, 5] = np.nan, np.inf
    for rotate in (True, False):
        y = w4.mxfp4_gemm(w4.mxfp4_rotate_quantize(f32_tensor(w, dev), rotate=rotate),
                          w4.mxfp4_rotate_quantize(f32_tensor(x, dev), rotate=rotate))
        want = torch.zeros(70, 150, dtype=torch.bool)
        want[66], want[:, 9] = True, True
        assert torch.equal(torch.isnan(y).cpu(), want)


def test_empty(dev):
    qw, qa = operands(dev, 4, 64, 8)
    assert w4.mxfp4_gemm(qw, w4.mxfp4_rotate_quantize(torch.zeros(0, 64, device=dev))).shape == (0, 8)
    assert w4.mxfp4_gemm(w4.mxfp4_rotate_quantize(torch.zeros(0, 64, device=dev)), qa).shape == (4, 0)


def test_refuses_mixed_rotation(dev):
    qw, _ = operands(dev, 4, 64, 8)
    _, qa = operands(dev, 4, 64, 8, rotate=False)
    with pytest.raises(w4.W4A4Error, match="MISMATCH"):
        w4.mxfp4_gemm(qw, qa)


def test_other_stream_and_graph(dev):
    qw, qa = operands(dev, 37, 736, 300)
    want = w4.mxfp4_gemm(qw, qa)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = w4.mxfp4_gemm(qw, qa, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    x = f32_tensor(rows(2, 37, 736), dev)
    q = w4.mxfp4_rotate_quantize(x)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.mxfp4_rotate_quantize(x, out=q)
        w4.mxfp4_gemm(qw, q, y=out)
    for scale in (1.0, 0.5):
        x.copy_(f32_tensor(rows(2, 37, 736), dev) * scale)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want * scale)


def test_offsets_past_32_bits(dev):
    """Inputs of 2^31 values and outputs of 2^31 values: the last rows repeat the first ones."""
    K, M = 17408, 126976  # 2.2e9 values
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    head = torch.from_numpy(rows(1, 130, K)).to(dev).to(torch.bfloat16)
    x[:130], x[-130:] = head, head
    q = w4.mxfp4_rotate_quantize(x)
    del x
    want = w4.mxfp4_rotate_quantize(head)
    assert torch.equal(q.codes[:130], want.codes) and torch.equal(q.codes[-130:], want.codes)
    sc = q.scales
    assert torch.equal(sc[-130:], want.scales)
    back = w4.mxfp4_dequantize(q, dtype=torch.bfloat16)
    assert torch.equal(back[-130:], w4.mxfp4_dequantize(want, dtype=torch.bfloat16))
    del back, q, sc
    N = 17000
    qw = w4.mxfp4_rotate_quantize(torch.from_numpy(rows(2, N, 64)).to(dev))
    xs = torch.zeros(M, 64, device=dev)
    xs[-130:] = torch.from_numpy(rows(3, 130, 64)).to(dev)
    y = w4.mxfp4_gemm(qw, w4.mxfp4_rotate_quantize(xs), dtype=torch.bfloat16)
    tail = w4.mxfp4_gemm(qw, w4.mxfp4_rotate_quantize(xs[-130:].contiguous()), dtype=torch.bfloat16)
    assert torch.equal(y[-130:], tail) and not bool(y[:-130].any())


@pytest.mark.parametrize("M,K,N", [(3, 2048, 640), (100, 512, 200), (600, 1024, 6000), (257, 8224, 10100)])
def test_wait_runs_out_then_recovers(dev, M, K, N):
    """A bounded pipeline wait that gives up (the copies held back longer than the bound): the kernel returns by
    itself, w4a4_check reports it, and the next call is right again.  Split and unsplit small tiles, pairs with whole
    tiles, pairs with their stages cut."""
    qw, qa = operands(dev, M, K, N)
    want = w4.mxfp4_gemm(qw, qa)
    w4.w4a4_check()
    try:
        w4.w4a4_debug_set_wait_limit(50_000, 5_000_000)
        w4.mxfp4_gemm(qw, qa)
        with pytest.raises(w4.W4A4Error, match="TIMEOUT"):
            w4.w4a4_check()
    finally:
        w4.w4a4_debug_set_wait_limit(0, 0)
    assert torch.equal(w4.mxfp4_gemm(qw, qa), want)
    w4.w4a4_check()
