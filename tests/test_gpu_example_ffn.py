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


def test_example_runs():
    out = subprocess.run([sys.executable, PATH, "--tokens", "64", "--hidden", "512", "--ffn", "1024"], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "us a block" in out.stdout, out.stdout + out.stderr
