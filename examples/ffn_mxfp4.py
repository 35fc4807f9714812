"""A feed-forward block in MXFP4: residual + RMS norm -> gate/up product -> SwiGLU -> down product.

    python examples/ffn_mxfp4.py [--tokens 512] [--hidden 5120] [--ffn 17408]

Weights and inputs are random.  Every step runs in the package's kernels: the norm writes the
MXFP4 operand of the gate/up product, SwiGLU that of the down product, and the rotations of
both operands cancel in each product.  Prints the block's time and its error against fp32.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import hadamard_rotated_w4a4_gb300 as w4  # noqa: E402


@dataclass
class FfnWeights:
    """A block's weights as the products take them (quantised once)."""
    gain: torch.Tensor    # [hidden], the norm's
    gate_up: w4.MxFp4     # [2 * ffn][hidden]: gate rows, then up rows
    down: w4.MxFp4        # [hidden][ffn]


def pack(gain: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor) -> FfnWeights:
    return FfnWeights(gain, w4.mxfp4_rotate_quantize(gate_up), w4.mxfp4_rotate_quantize(down))


def ffn(x: torch.Tensor, residual: torch.Tensor, w: FfnWeights, eps: float = 1e-6) -> torch.Tensor:
    """The block's output [tokens][hidden] (bf16), to be added to `residual` by the next norm.

    x: the layer before's output; it is added to `residual` in place.
    """
    a = w4.mxfp4_rmsnorm_quantize(x, w.gain, eps=eps, residual=residual)
    gu = w4.mxfp4_gemm(w.gate_up, a, dtype=torch.bfloat16)
    f = gu.shape[1] // 2
    return w4.mxfp4_gemm(w.down, w4.mxfp4_swiglu_quantize(gu[:, :f], gu[:, f:]), dtype=torch.bfloat16)


def ffn_fp32(x, residual, gain, gate_up, down, eps: float = 1e-6) -> torch.Tensor:
    """The same block in fp32, unquantised."""
    h = x.float() + residual.float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * gain
    g, u = (y @ gate_up.float().T).chunk(2, dim=1)
    return (g / (1 + torch.exp(-g)) * u) @ down.float().T


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--ffn", type=int, default=17408)
    a = ap.parse_args()
    w4.load_library(build_if_missing=True)
    gen = torch.Generator("cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    gate_up, down = ((randn(*s) * 0.02).bfloat16() for s in ((2 * a.ffn, a.hidden), (a.hidden, a.ffn)))
    gain = 1 + 0.1 * randn(a.hidden)
    x, r = randn(a.tokens, a.hidden).bfloat16(), randn(a.tokens, a.hidden).bfloat16()
    w = pack(gain, gate_up, down)
    want = ffn_fp32(x, r, gain, gate_up, down)
    got = ffn(x, r.clone(), w).float()
    w4.w4a4_check()
    print(f"relative error against fp32: {float((got - want).norm() / want.norm()):.3f}")

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        ffn(x, r, w)  # the workspace of this stream
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(10):
            ffn(x, r, w)
    graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record()
    graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 100
    flops = 6 * a.tokens * a.hidden * a.ffn
    print(f"{a.tokens} tokens, hidden {a.hidden}, ffn {a.ffn}: {us:.1f} us a block, {flops / us * 1e-6:.0f} TFLOP/s")


if __name__ == "__main__":
    main()
