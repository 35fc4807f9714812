"""The example's feed-forward block against the same chain in 64 bits with the oracle's quantiser."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from w4a4_testutil import device

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "ffn_mxfp4.py")


def rounded(v):
    """fp64 -> bf16 -> fp64."""
    return torch.from_numpy(v.astype(np.float32)).bfloat16().double().numpy()


@pytest.mark.parametrize("M,H,F", [(1, 256, 384), (33, 416, 736), (200, 512, 1024)])
def test_block_matches_the_chain(M, H, F):
    dev = device()
    spec = importlib.util.spec_from_file_location("ffn_mxfp4", PATH)
    ex = importlib.util.module_from_spec(spec)
    sys.modules["ffn_mxfp4"] = ex
    spec.loader.exec_module(ex)
    rng = np.random.default_rng(H)
    x, r, gu, dn = (rounded(rng.standard_normal(s) * k) for s, k in
                    (((M, H), 1), ((M, H), 1), ((2 * F, H), 0.02), ((H, F), 0.02)))
    g = (1 + 0.1 * rng.standard_normal(H)).astype(np.float32)
    t = lambda v: torch.from_numpy(v.astype(np.float32)).to(dev).bfloat16()  # noqa: E731
    res = t(r)
    got = ex.ffn(t(x), res, ex.pack(torch.from_numpy(g).to(dev), t(gu), t(dn))).double().cpu().numpy()
    assert torch.equal(res, t(x + r))  # the residual stream was updated in place

    def q(v):
        m = oracle.quantize_mxfp4(v.astype(np.float32))
        return oracle.mxfp4_values(m["codes"], m["scales"])

    h = x + r
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + 1e-6) * g
    p = rounded(q(y) @ q(gu).T)
    want = q(p[:, :F] / (1 + np.exp(-p[:, :F])) * p[:, F:]) @ q(dn).T
    # bf16 outputs (2^-8), and the odd code that moves by a step where fp32 sits on a boundary
    assert np.linalg.norm(got - want) <= 0.02 * np.linalg.norm(want)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_chain_without_waits_between(M):
    """Kernels may start before the one in front of them ends and share their buffers with it: a hundred blocks
    in a row, every buffer reused, give the bits of the same blocks with a wait behind each call."""
    import hadamard_rotated_w4a4_gb300 as w4

    dev = device()
    H, F = 512, 768
    gen = torch.Generator("cuda").manual_seed(M)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    wg, wd = w4.mxfp4_rotate_quantize(rnd(2 * F, H) * 0.04), w4.mxfp4_rotate_quantize(rnd(H, F) * 0.04)
    x0, r0 = rnd(M, H).bfloat16(), rnd(M, H).bfloat16()

    def blocks(wait):
        x, r = x0.clone(), r0.clone()
        a, b = w4.MxFp4(M, H, dev), w4.MxFp4(M, F, dev)
        gu = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=dev)
        for _ in range(100):
            for call in (lambda: w4.mxfp4_rmsnorm_quantize(x, residual=r, out=a), lambda: w4.mxfp4_gemm(wg, a, y=gu),
                         lambda: w4.mxfp4_swiglu_quantize(gu[:, :F], gu[:, F:], out=b),
                         lambda: w4.mxfp4_gemm(wd, b, y=x)):
                call()
                if wait:
                    torch.cuda.synchronize()
        return x, r

    want, got = blocks(True), blocks(False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bool(torch.isfinite(got[1]).all())


def test_example_runs():
    out = subprocess.run([sys.executable, PATH, "--tokens", "64", "--hidden", "512", "--ffn", "1024"], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "us a block" in out.stdout, out.stdout + out.stderr
