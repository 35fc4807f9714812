"""A transformer layer in MXFP4 over an 8-bit paged KV cache: prompts of several lengths, then a token at a time.

    python examples/layer_mxfp4.py [--hidden 5120] [--q-heads 40] [--kv-heads 8] [--dim 128] [--ffn 17408] [--batch 16]
                                   [--prompt 1000] [--steps 32]

Weights and inputs are random.  RMS norm -> q, k, v product + bias -> positions and append to the cache -> attention over
its pages -> output product + residual -> RMS norm -> up product, GELU -> down product + residual.  Every step runs in the
package's kernels, and tables and lengths stay on the GPU: one captured graph serves every step of a token each.
Prints the time of the prompts and of a step, and the layer's error against fp32 on the first prompt.
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
class LayerWeights:
    """A layer's weights as the products take them (quantised once)."""
    norm1: torch.Tensor   # [hidden]
    qkv: w4.MxFp4         # [(q_heads + 2 kv_heads) * dim][hidden]
    qkv_bias: torch.Tensor
    out: w4.MxFp4         # [hidden][q_heads * dim]
    norm2: torch.Tensor   # [hidden]
    up: w4.MxFp4          # [ffn][hidden]
    up_bias: torch.Tensor
    down: w4.MxFp4        # [hidden][ffn]
    freqs: torch.Tensor   # [dim / 2] fp64


def pack(norm1, qkv, qkv_bias, out, norm2, up, up_bias, down, freqs) -> LayerWeights:
    q = w4.mxfp4_rotate_quantize
    return LayerWeights(norm1, q(qkv), qkv_bias, q(out), norm2, q(up), up_bias, q(down), freqs)


def layer(h: torch.Tensor, w: LayerWeights, cache: w4.KvCache8, table: torch.Tensor, lens: torch.Tensor,
          cu: torch.Tensor | None = None, window: int = 0) -> torch.Tensor:
    """The layer on new tokens h [tokens][hidden] (bf16, the residual stream), in place; their keys and values join the cache.

    table, lens (the new tokens included) and cu as kv8_append takes them.
    """
    T, heads, D = h.shape[0], cache.heads, cache.dim
    qkv = w4.mxfp4_gemm_epilogue(w.qkv, w4.mxfp4_rmsnorm_quantize(h, w.norm1), w.qkv_bias, dtype=torch.bfloat16).view(T, -1, D)
    q, k, v = qkv.split([qkv.shape[1] - 2 * heads, heads, heads], dim=1)
    w4.kv8_append(cache, k, v, table, lens, cu, q=q, freqs=w.freqs)
    o = w4.kv8_attention(q, cache, table, lens, cu, window=window).view(T, -1)
    w4.mxfp4_gemm_epilogue(w.out, w4.mxfp4_rotate_quantize(o), residual=h, y=h)
    u = w4.mxfp4_gemm_epilogue(w.up, w4.mxfp4_rmsnorm_quantize(h, w.norm2), w.up_bias, "gelu", dtype=torch.bfloat16)
    return w4.mxfp4_gemm_epilogue(w.down, w4.mxfp4_rotate_quantize(u), residual=h, y=h)


def layer_fp32(h, norm1, qkv, qkv_bias, out, norm2, up, up_bias, down, freqs, kv_heads: int) -> torch.Tensor:
    """The same layer on one whole sequence in fp32, unquantised."""
    def norm(x, g):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * g

    h = h.float()
    T, n = h.shape[0], freqs.shape[0]
    a = torch.outer(torch.arange(T, device=h.device, dtype=torch.float64), freqs)
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]

    def turn(x):
        return torch.cat([x[..., :n] * c - x[..., n:] * s, x[..., n:] * c + x[..., :n] * s], dim=-1)

    x = (norm(h, norm1) @ qkv.float().T + qkv_bias).view(T, -1, 2 * n)
    q, k, v = x.split([x.shape[1] - 2 * kv_heads, kv_heads, kv_heads], dim=1)
    o = torch.nn.functional.scaled_dot_product_attention(
        *(t.transpose(0, 1) for t in (turn(q), turn(k), v)), is_causal=True, enable_gqa=True).transpose(0, 1).reshape(T, -1)
    h = h + o @ out.float().T
    return h + torch.nn.functional.gelu(norm(h, norm2) @ up.float().T + up_bias) @ down.float().T


def main() -> None:
    ap = argparse.ArgumentParser()
    for name, value in (("hidden", 5120), ("q-heads", 40), ("kv-heads", 8), ("dim", 128), ("ffn", 17408), ("batch", 16),
                        ("prompt", 1000), ("steps", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    w4.load_library(build_if_missing=True)
    gen = torch.Generator("cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    raw = (1 + 0.1 * randn(a.hidden), (randn((a.q_heads + 2 * a.kv_heads) * a.dim, a.hidden) * 0.02).bfloat16(),
           0.1 * randn((a.q_heads + 2 * a.kv_heads) * a.dim), (randn(a.hidden, a.q_heads * a.dim) * 0.02).bfloat16(),
           1 + 0.1 * randn(a.hidden), (randn(a.ffn, a.hidden) * 0.02).bfloat16(), 0.1 * randn(a.ffn),
           (randn(a.hidden, a.ffn) * 0.02).bfloat16(), w4.rope_freqs(a.dim))
    w = pack(*raw)

    # prompts of a quarter of the length and up; pages for them and the steps, in any order
    counts = [max(1, a.prompt * (4 - b % 4) // 4) for b in range(a.batch)]
    page = 64
    width = (a.prompt + a.steps + page - 1) // page
    table = torch.randperm(a.batch * width, device="cuda", generator=gen).int().view(a.batch, width)
    cache = w4.alloc_kv8(a.batch * width, a.kv_heads, a.dim, page)
    lens = torch.tensor(counts, dtype=torch.int32, device="cuda")
    cu = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).int()
    x = randn(sum(counts), a.hidden).bfloat16()

    want = layer_fp32(x[:counts[0]], *raw, a.kv_heads)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    layer(x.clone(), w, cache, table, lens, cu)  # a second time below: the same tokens, so the same pages
    h = x.clone()
    torch.cuda.synchronize()
    begin.record()
    layer(h, w, cache, table, lens, cu)
    end.record()
    w4.w4a4_check()
    off, y = h[:counts[0]].float() - want, want - x[:counts[0]].float()
    print(f"relative error against fp32: {float(off.norm() / y.norm()):.3f}")
    print(f"{sum(counts)} tokens of {a.batch} prompts: {begin.elapsed_time(end) * 1000:.0f} us")

    token = randn(a.batch, a.hidden).bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        layer(token, w, cache, table, lens)
    graph.replay()
    torch.cuda.synchronize()
    begin.record()
    for _ in range(a.steps - 1):
        graph.replay()
    end.record()
    w4.w4a4_check()
    print(f"{a.batch} sequences, a token each: {begin.elapsed_time(end) * 1000 / max(1, a.steps - 1):.1f} us a step")


if __name__ == "__main__":
    main()
