"""Shared by the kv8 GPU tests: caches of known content, and attention in 64 bits with the bound
of what the kernels may be off by."""
from __future__ import annotations

import numpy as np
import torch

import hadamard_rotated_w4a4_gb300 as w4
import oracle

U = 2.0 ** -24


def make_cache(rng, dev, pages, heads, page, dim, rotated=True, spread=3):
    """Random codes and scales (a few powers of two apart) on the GPU, and on the host."""
    codes = rng.integers(-127, 128, (pages, heads, 2, page, dim)).astype(np.int8)
    scales = (127 - 6 + rng.integers(-spread, 1, (pages, heads, 2, page // 16))).astype(np.uint8)
    scales[:, :, 0] -= 1  # keys of a size that leaves the softmax some width
    return w4.KvCache8(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), rotated), codes, scales


def make_table(rng, dev, pages, lens, page, width=None):
    """Distinct random pages for each sequence; entries past its length are -1 (never looked at)."""
    need = [(L + page - 1) // page for L in lens]
    width = max(need + [1]) if width is None else width
    ids = rng.permutation(pages)
    t, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, torch.from_numpy(t).to(dev)


def ints(x, dev):
    return torch.tensor(list(x), dtype=torch.int32, device=dev)


def values(codes, scales, table_row, L):
    """[2][L][H][D] fp64."""
    page = codes.shape[3]
    pids = table_row[: (L + page - 1) // page]
    s = scales[pids].astype(np.float64)
    s = np.repeat(np.where(s == 255, np.nan, 2.0 ** (s - 127)), 16, axis=-1)
    x = codes[pids].astype(np.float64) * s[..., None]  # [P][H][2][page][D]
    return x.transpose(2, 0, 3, 1, 4).reshape(2, -1, codes.shape[1], codes.shape[4])[:, :L]


def attention_64(q, k, v, scale, causal, window, rotated):
    """One sequence: q [n][Hq][D] (fp64), k, v [L][H][D] as stored; the result, and by how much a kernel's fp32
    result may miss it, before its rounding to the output's type.

    q, scaled by a power of two: fp16, half a step 2^-11 relative (2^-25 of the smallest step, 2^-24, where the row's largest is 2^7 or
    more: 2^-32 of it absolute); with the rotation 6 fp32 roundings on 32 B / sqrt 32 = 5.66 B, under 40 U of the
    block's largest.  Products with the codes are exact, D of them summed in fp32: D U of sum |q k|.  Score in log2:
    scale, fused multiply and subtraction, 4 U of itself and of numbers up to |t| + 64.  A weight: exp2 2 ulp, 2^-22,
    and fp16, 2^-11 relative or 2^-29 of the row's largest; sums of L weights and of L products in fp32, L U each at
    most, rescaled once per block of 16: L / 16 roundings more.  What a score is off by moves the weights by
    exp(2 d) - 1 against each other.
    """
    n, Hq, D = q.shape
    L, H, _ = k.shape
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    if L == 0:
        return out, tol
    g = Hq // H
    qs = oracle.rotate_h32(q, dtype=np.float64) if rotated else q
    pos, key = np.arange(L - n, L)[:, None], np.arange(L)
    see = (key <= pos) if causal else np.ones((n, L), bool)
    if window:
        see &= key > pos - window
    amax = np.abs(qs).max(axis=-1, keepdims=True)
    dq = 2.0 ** -11 * np.abs(qs) + 2.0 ** -32 * amax + (40 * U * amax if rotated else 0)
    for h in range(Hq):
        K, V = k[:, h // g], v[:, h // g]
        s = scale * (qs[:, h] @ K.T)
        mag = abs(scale) * (np.abs(qs[:, h]) @ np.abs(K).T)
        d = abs(scale) * (dq[:, h] @ np.abs(K).T) + (D + 8) * U * mag + 300 * U
        s = np.where(see, s, -np.inf)
        top = s.max(axis=1, keepdims=True)
        w = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0)), 0.0)
        tot = w.sum(axis=1, keepdims=True)
        some = tot[:, 0] > 0
        p = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
        out[:, h] = p @ V
        rel = np.expm1(2 * np.where(see, d, 0).max(axis=1, keepdims=True)) + 2.0 ** -11 + 2.0 ** -20 + (L + L / 8) * U
        tiny = 2.0 ** -29 * np.divide(1, tot, out=np.zeros_like(tot), where=tot > 0)
        tol[:, h] = (rel * p + tiny * see) @ np.abs(V) * some[:, None]
    if rotated:  # the inverse rotation of the result, and its own roundings
        out = oracle.rotate_h32(out, dtype=np.float64)
        b = tol.reshape(n, Hq, D // 32, 32)
        tol = np.repeat(b.sum(-1, keepdims=True) / np.sqrt(32), 32, axis=-1).reshape(tol.shape)
        tol += 40 * U * np.abs(out).max(axis=-1, keepdims=True)
    return out, tol


def check_attention(got, q, codes, scales, table, lens, counts, scale=None, causal=True, window=0, rotated=True):
    """got, q: torch [T][Hq][D]; every sequence's tokens against attention_64."""
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    eps = torch.finfo(got.dtype).eps / 2
    got, q = got.double().cpu().numpy(), q.double().cpu().numpy()
    t = 0
    for b, (L, n) in enumerate(zip(lens, counts)):
        k, v = values(codes, scales, table[b], L)
        want, tol = attention_64(q[t:t + n], k, v, scale, causal, window, rotated)
        off = np.abs(got[t:t + n] - want) - tol - eps * (np.abs(want) + tol)
        assert not np.isnan(got[t:t + n]).any(), f"sequence {b}: NaN"
        assert (off <= 0).all(), (f"sequence {b} of {L} keys, {n} tokens: off by {np.abs(got[t:t + n] - want).max():.3e}, "
                                  f"allowed {tol.max():.3e}, first at {np.argwhere(off > 0)[0]}")
        t += n
