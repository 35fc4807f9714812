"""Keys and values in 8 bits, in pages -- oracle side: appending, reading back, attention.

Pages of ``page`` tokens; of each page and head the keys, then the values, as int8 codes;
16 tokens of a head share a scale 2^(s - 127), one for K and one for V.  Token t of
sequence b stands in page ``table[b][t // page]`` at row ``t % page``.

Append, per (block of 16 tokens, head, K or V) that gets new rows y (fp32, after the
rotary rotation of K and the optional H32 rotation): E = the least integer with
max |y| <= 127 * 2^E, clamped to -40..40 (-40 where all are zero).  If older rows stand in
the block, whose scale is 2^F: E becomes max(E, F) and the older codes q become
rint(q 2^(F - E)).  New codes: rint(y 2^-E), clamped to +-127.  An infinity or a NaN among
the new rows, or scale byte 255 over older rows: byte 255 and new codes of zero.
"""
from __future__ import annotations

import numpy as np

KV8_TOKENS = 16
KV8_LOW, KV8_HIGH = -40, 40


def rope(x: np.ndarray, pos: np.ndarray, freqs: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [T][H][D] in 64 bits, pair i turned by pos * freqs[i]: pairs (i, i + n), or (2i, 2i + 1)."""
    x = np.array(x, dtype=np.float64)
    n = len(freqs)
    a = pos[:, None].astype(np.float64) * freqs
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    u, v = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo], x[..., hi] = u * c - v * s, v * c + u * s
    return x


def kv8_exponent(amax: float) -> int:
    """The least E with amax <= 127 * 2^E, in KV8_LOW..KV8_HIGH."""
    E = KV8_LOW
    while E < KV8_HIGH and amax > 127 * 2.0 ** E:
        E += 1
    return E


def kv8_append(codes: np.ndarray, scales: np.ndarray, k: np.ndarray, v: np.ndarray, table: np.ndarray, lens, counts) -> None:
    """In place; k, v [T][H][D] as they are to be stored (rotations done)."""
    page = codes.shape[3]
    t = 0
    for b, (L, n) in enumerate(zip(lens, counts)):
        for p0 in range((L - n) // KV8_TOKENS * KV8_TOKENS, L, KV8_TOKENS):
            lo, hi = max(L - n - p0, 0), min(L - p0, KV8_TOKENS)
            if n == 0:
                continue
            pid, row = table[b][p0 // page], p0 % page
            for h in range(codes.shape[1]):
                for kind, x in ((0, k), (1, v)):
                    y = x[t + p0 + lo - (L - n): t + p0 + hi - (L - n), h].astype(np.float64)
                    was = int(scales[pid, h, kind, row // KV8_TOKENS]) if lo else None
                    if not np.isfinite(y).all() or was == 255:
                        scales[pid, h, kind, row // KV8_TOKENS] = 255
                        codes[pid, h, kind, row + lo: row + hi] = 0
                        continue
                    E = kv8_exponent(np.abs(y).max())
                    if lo:
                        F = was - 127
                        E = max(E, F)
                        old = codes[pid, h, kind, row: row + lo].astype(np.float64)
                        codes[pid, h, kind, row: row + lo] = np.rint(old * 2.0 ** (F - E)).astype(np.int8)
                    codes[pid, h, kind, row + lo: row + hi] = np.clip(np.rint(y * 2.0 ** -E), -127, 127).astype(np.int8)
                    scales[pid, h, kind, row // KV8_TOKENS] = E + 127
        t += n


def kv8_values(codes: np.ndarray, scales: np.ndarray, pages, length: int) -> np.ndarray:
    """The values of a sequence's first `length` tokens, fp64 [2][length][H][D] (K, then V)."""
    page = codes.shape[3]
    out = np.zeros((2, length, codes.shape[1], codes.shape[4]))
    for t in range(length):
        pid, row = pages[t // page], t % page
        s = scales[pid, :, :, row // KV8_TOKENS].astype(np.float64)
        s = np.where(s == 255, np.nan, 2.0 ** (s - 127))
        out[:, t] = (codes[pid, :, :, row].astype(np.float64) * s[..., None]).swapaxes(0, 1)
    return out


def kv8_attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool, window: int) -> np.ndarray:
    """One sequence in 64 bits: q [n][Hq][D], its last n tokens; k, v [L][H][D]; tokens that see nothing get zeros."""
    n, Hq, _ = q.shape
    L, H, _ = k.shape
    out = np.zeros(q.shape)
    for i in range(n):
        pos = L - n + i
        hi = min(L, pos + 1) if causal else L
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            g = h // (Hq // H)
            s = scale * (k[lo:hi, g] @ q[i, h].astype(np.float64))
            w = np.exp(s - s.max())
            out[i, h] = w @ v[lo:hi, g] / w.sum()
    return out
