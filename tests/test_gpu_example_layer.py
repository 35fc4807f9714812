"""The example's layer, prompts and then single tokens over the same cache: each of its calls against 64 bits; the same calls
without waits between them; the example's run."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
import oracle
from kv8_testutil import U, check_attention, ints, make_table
from test_gpu_epilogue import check
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "layer_mxfp4.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("layer_mxfp4", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules["layer_mxfp4"] = m
    spec.loader.exec_module(m)
    return m


def rounded(v):
    """fp64 -> bf16 -> fp64."""
    return torch.from_numpy(v.astype(np.float32)).bfloat16().double().numpy()


def norm(x, g):
    return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + 1e-6) * g


def check_operand(a, y):
    """The MXFP4 operand of rows y (fp64): no element further from H32 y than a quarter of its block's largest magnitude a, as
    e2m1 of a scale 2^E with 4 2^E <= a < 8 2^E has gaps of 2 2^E at most and ends at 6 2^E; fp32 on the way: 2^-10 of that."""
    y = oracle.rotate_h32(y, dtype=np.float64).reshape(y.shape[0], -1, 32)
    got = w4.mxfp4_dequantize(a).double().cpu().numpy().reshape(y.shape)
    assert (np.abs(got - y) <= np.abs(y).max(axis=-1, keepdims=True) * 0.25 * (1 + 2.0 ** -10)).all()


def random_weights(rng, H, Hq, Hkv, D, F):
    n = (Hq + 2 * Hkv) * D
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    return [(1 + 0.1 * f(H)).astype(np.float32), rounded(f(n, H) * 0.04), (0.1 * f(n)).astype(np.float32), rounded(f(H, Hq * D) * 0.04),
            (1 + 0.1 * f(H)).astype(np.float32), rounded(f(F, H) * 0.04), (0.1 * f(F)).astype(np.float32), rounded(f(H, F) * 0.04),
            10000.0 ** (-np.arange(0, D, 2) / D)]


def on_gpu(ex, w, dev):
    types = (torch.float32, torch.bfloat16, torch.float32, torch.bfloat16, torch.float32, torch.bfloat16, torch.float32, torch.bfloat16,
             torch.float64)
    return ex.pack(*(torch.from_numpy(np.ascontiguousarray(v)).to(dev).to(t) for v, t in zip(w, types)))


@pytest.mark.parametrize("H,Hq,Hkv,D,F,page,counts,window,rotated", [
    (256, 4, 2, 128, 384, 16, [40, 3, 61], 0, True), (384, 6, 1, 64, 480, 32, [9, 1, 70], 24, True),
    (256, 2, 2, 256, 256, 64, [33, 20], 0, False)])
def test_layer_step_by_step(ex, H, Hq, Hkv, D, F, page, counts, window, rotated):
    """Prompts, then three steps of a token each: every call of the layer on what the call before gave, against 64 bits;
    the example's layer gives the same bits, and leaves the same cache."""
    dev = device()
    rng = np.random.default_rng(D)
    w = random_weights(rng, H, Hq, Hkv, D, F)
    wg = on_gpu(ex, w, dev)
    B, total = len(counts), max(counts) + 3
    pages = B * (total // page + 1)
    table, t = make_table(rng, dev, pages, [total] * B, page)
    cache, other = (w4.alloc_kv8(pages, Hkv, D, page, dev, rotated) for _ in range(2))
    lens, new = [0] * B, counts
    for step in range(4):
        lens = [L + n for L, n in zip(lens, new)]
        T = sum(new)
        h = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dev).bfloat16()
        cu, glens = None if step else ints([0] + list(np.cumsum(new)), dev), ints(lens, dev)
        as64 = lambda x: x.double().cpu().numpy()  # noqa: E731

        a = w4.mxfp4_rmsnorm_quantize(h, wg.norm1)
        check_operand(a, norm(as64(h), w[0].astype(np.float64)))
        x = w4.mxfp4_gemm_epilogue(wg.qkv, a, wg.qkv_bias, dtype=torch.bfloat16)
        check(x, w4.mxfp4_gemm(wg.qkv, a), wg.qkv_bias, None, None)

        q, k, v = x.view(T, -1, D).split([Hq, Hkv, Hkv], dim=1)
        q_in = as64(q)
        w4.kv8_append(cache, k, v, t, glens, cu, q=q, freqs=wg.freqs)
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
        turned, B_q = oracle.rope(q_in, pos, w[8], False), np.abs(q_in).max(axis=-1, keepdims=True)
        assert (np.abs(as64(q) - turned) <= 2.0 ** -8 * np.abs(turned) + 20 * U * B_q).all()
        back = w4.kv8_read(cache, t, glens, T, cu)
        scales, at = cache.scales.cpu().numpy(), 0
        for b, (L, n) in enumerate(zip(lens, new)):
            p = np.arange(L - n, L)
            for kind, (got, y) in enumerate(zip(back, (oracle.rope(as64(k)[at:at + n], p, w[8], False), as64(v)[at:at + n]))):
                unit = 2.0 ** (scales[table[b][p // page], :, kind, p % page // 16].astype(np.float64) - 127)[..., None]
                big = np.abs(y).max(axis=-1, keepdims=True)
                y = oracle.rotate_h32(y, dtype=np.float64) if rotated else y  # an angle's and H32's roundings: 160 U
                assert (np.abs(as64(got)[at:at + n] - y) <= unit / 2 + 160 * U * big).all()
            at += n

        o = w4.kv8_attention(q, cache, t, glens, cu, window=window)
        check_attention(o, q, cache.codes.cpu().numpy(), scales, table, lens, new, window=window, rotated=rotated)
        a = w4.mxfp4_rotate_quantize(o.view(T, -1))
        check_operand(a, as64(o).reshape(T, -1))
        h2 = w4.mxfp4_gemm_epilogue(wg.out, a, residual=h, dtype=torch.bfloat16)
        check(h2, w4.mxfp4_gemm(wg.out, a), None, None, h)

        a = w4.mxfp4_rmsnorm_quantize(h2, wg.norm2)
        check_operand(a, norm(as64(h2), w[4].astype(np.float64)))
        u = w4.mxfp4_gemm_epilogue(wg.up, a, wg.up_bias, "gelu", dtype=torch.bfloat16)
        check(u, w4.mxfp4_gemm(wg.up, a), wg.up_bias, "gelu", None)
        a = w4.mxfp4_rotate_quantize(u)
        check_operand(a, as64(u))
        h3 = w4.mxfp4_gemm_epilogue(wg.down, a, residual=h2, dtype=torch.bfloat16)
        check(h3, w4.mxfp4_gemm(wg.down, a), None, None, h2)

        assert ex.layer(h, wg, other, t, glens, cu, window) is h
        assert torch.equal(h, h3) and torch.equal(other.codes, cache.codes) and torch.equal(other.scales, cache.scales)
        new = [1] * B
    w4.w4a4_check()


@pytest.mark.parametrize("B", [1, 7])
def test_layers_without_waits_between(ex, B):
    """Kernels may start before the one in front of them ends: a prompt and thirty steps of two layers over the same
    buffers give the bits of the same calls with a wait behind each; so does a captured step that is replayed."""
    dev = device()
    rng = np.random.default_rng(B)
    H, Hq, Hkv, D, page, n, steps = 512, 8, 2, 128, 64, 50, 30
    layers = [on_gpu(ex, random_weights(rng, H, Hq, Hkv, D, 768), dev) for _ in range(2)]
    pages = 2 * B
    t = ints(rng.permutation(pages), dev).view(B, 2)
    x = [torch.from_numpy(rng.standard_normal((B * k, H)).astype(np.float32)).to(dev).bfloat16() for k in (n, 1)]

    def run(how):
        caches = [w4.alloc_kv8(pages, Hkv, D, page, dev) for _ in layers]
        lens = torch.full((B,), n, dtype=torch.int32, device=dev)
        h, token = x[0].clone(), x[1].clone()

        def all_layers(h):
            for w, c in zip(layers, caches):
                ex.layer(h, w, c, t, lens)
                if how == "waits":
                    torch.cuda.synchronize()

        all_layers(h)
        if how == "graph":
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                lens += 1
                all_layers(token)
            for _ in range(steps):
                graph.replay()
        else:
            for _ in range(steps):
                lens += 1
                all_layers(token)
        w4.w4a4_check()
        return [h, token] + [y for c in caches for y in (c.codes, c.scales)]

    want = run("waits")
    assert all(bool(torch.isfinite(y).all()) for y in want[:2])
    for how in ("no waits", "graph"):
        assert all(torch.equal(a, b) for a, b in zip(run(how), want)), how


def test_example_runs():
    out = subprocess.run([sys.executable, PATH, "--hidden", "512", "--q-heads", "4", "--kv-heads", "2", "--ffn", "1024", "--batch", "3",
                          "--prompt", "90", "--steps", "4"], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "us a step" in out.stdout, out.stdout + out.stderr
