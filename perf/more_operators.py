"""Measured cases of the attention half of a layer: the 8-bit paged key/value cache, attention
over it, and the MXFP4 product with bias, activation and residual.

``run`` computes each operator either with elementary torch operations in 32 bits
(``own`` false) or with the package's entry points (``own`` true):

* ``append``:  rotary positions on q and k, H32 rotation of k and v, int8 with one power-of-two
               scale per 16 tokens and head into the pages, the touched blocks read back;
* ``attend``:  attention of new tokens over the pages, from single tokens to long prompts;
* ``product``: MXFP4 weights times MXFP4 activations, then bias, activation and residual.

Shapes are those of the package's workloads (hidden 5120 as 40 heads of 128 or 20 of 256, FFN
17408, 512- and 1024-token batches, 8-token verification batches) and generic ones between.
"""
import math
import random

import torch

own = False

BLOCK = 32      # elements of a rotation block and of an MXFP4 block
TOKENS = 16     # tokens that share a cache scale
LOW, TOP = -40, 40  # exponents that a cache scale may have
BASE = 1e6      # rotary base
C_H32 = 0.1767766922712326  # fl32(1 / sqrt 32)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


# ----------------------------------------------------------------- cases
# count: new tokens of a sequence; length: tokens it has with them; ragged: 0 = every sequence has
# just these, else the seed of sequences between a few tokens and these.
def listed():
    gqa = {"Hq": 40, "Hkv": 8, "D": 128, "rotate": True}
    return [
        # one sequence's next token: its heads after the qkv product, each decode step
        {"name": "append_token", "op": "append", "B": 1, "count": 1, "length": 1000, "ragged": 0, "page": 64,
         "interleaved": False, "dtype": "bf16", **gqa},
        # a served batch's next tokens, sequences of unlike lengths
        {"name": "append_batch", "op": "append", "B": 64, "count": 1, "length": 4096, "ragged": 3, "page": 16,
         "interleaved": True, "dtype": "f32", "Hq": 20, "Hkv": 4, "D": 256, "rotate": True},
        # a long prompt's keys and values
        {"name": "append_prompt", "op": "append", "B": 1, "count": 8192, "length": 8192, "ragged": 0, "page": 64,
         "interleaved": False, "dtype": "bf16", **gqa},
        # one sequence's next token over a short context, each decode step
        {"name": "attend_token", "op": "attend", "B": 1, "count": 1, "length": 1000, "ragged": 0, "page": 64,
         "causal": True, "window": 0, **gqa},
        # a served batch's next tokens, sequences of unlike lengths
        {"name": "attend_batch", "op": "attend", "B": 64, "count": 1, "length": 8192, "ragged": 5, "page": 16,
         "causal": True, "window": 0, **gqa},
        # next tokens of a few long documents
        {"name": "attend_long", "op": "attend", "B": 4, "count": 1, "length": 131072, "ragged": 0, "page": 128,
         "causal": True, "window": 0, **gqa},
        # verification batches of eight drafted tokens, heads of 256
        {"name": "attend_verify", "op": "attend", "B": 8, "count": 8, "length": 6000, "ragged": 9, "page": 32,
         "causal": True, "window": 0, "Hq": 20, "Hkv": 4, "D": 256, "rotate": True},
        # ragged prompts of a smaller model with a sliding window, not rotated
        {"name": "attend_ragged", "op": "attend", "B": 7, "count": 777, "length": 2500, "ragged": 11, "page": 16,
         "causal": True, "window": 500, "Hq": 12, "Hkv": 4, "D": 64, "rotate": False},
        # a 4096-token piece of a long prompt behind 12288 tokens
        {"name": "attend_prompt", "op": "attend", "B": 1, "count": 4096, "length": 16384, "ragged": 0, "page": 64,
         "causal": True, "window": 0, **gqa},
        # one token through the qkv projection with its bias
        {"name": "product_qkv", "op": "product", "M": 1, "K": 5120, "N": 7168, "bias": True, "act": "none",
         "residual": "none", "out": "bf16"},
        # a ragged prompt tail through an up projection with bias and GELU
        {"name": "product_up", "op": "product", "M": 333, "K": 1184, "N": 4600, "bias": True, "act": "gelu",
         "residual": "none", "out": "bf16"},
        # a 1024-token micro-batch through the FFN down projection, added to the residual stream
        {"name": "product_down", "op": "product", "M": 1024, "K": 17408, "N": 5120, "bias": False, "act": "none",
         "residual": "f32", "out": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "product"))
    if op == "product":
        K = rng.choice((160 * _log(rng, 1, 108), BLOCK * (2 * _log(rng, 1, 271) + 1)))
        N = _log(rng, 64, 17408)
        M = _log(rng, 1, max(1, min(4096, 1024 * 17408 * 5120 // (N * K))))
        return {"op": op, "M": M, "K": K, "N": N, "bias": rng.random() < 0.6, "act": rng.choice(("none", "silu", "gelu", "gelu_tanh", "relu")),
                "residual": rng.choice(("none", "bf16", "f32")), "out": rng.choice(("f32", "bf16"))}
    D, Hkv = rng.choice((64, 128, 128, 256)), rng.randint(1, 8)
    c = {"op": op, "Hq": Hkv * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16)), "Hkv": Hkv, "D": D, "rotate": rng.random() < 0.7,
         "page": rng.choice((16, 32, 64, 128))}
    if op == "append":
        B = _log(rng, 1, 64)
        c["dtype"] = rng.choice(("bf16", "f32"))
        most = 8192 * 56 * 128 // (B * (c["Hq"] + 2 * Hkv) * D * (2 if c["dtype"] == "f32" else 1))
        c["count"] = rng.choice((1, _log(rng, 1, max(1, min(8192, most)))))
        c["length"] = c["count"] + rng.choice((0, _log(rng, 1, 4096)))
        c.update(B=B, ragged=rng.choice((0, rng.randint(1, 10**6))), interleaved=rng.random() < 0.3)
        return c
    B = _log(rng, 1, 64)
    keys = 4 * 131072 * 8 * 128 // (B * Hkv * D)
    c["count"] = rng.choice((1, rng.randint(2, 8), _log(rng, 9, 4096)))
    room = 40 * 4096 * 16384 * 128 // (B * c["Hq"] * c["count"] * max(D, 128))
    c["length"] = _log(rng, min(64, keys, room), max(64, min(131072, keys, room)))
    c["count"] = min(c["count"], c["length"])
    c.update(B=B, ragged=rng.choice((0, rng.randint(1, 10**6))), causal=rng.random() < 0.8)
    c["window"] = _log(rng, 1, c["length"]) if c["causal"] and rng.random() < 0.3 else 0
    return c


def _lengths(case):
    """Tokens of each sequence, and how many of them are new."""
    B, n, L = case["B"], case["count"], case["length"]
    if not case["ragged"]:
        return [L] * B, [n] * B
    r = random.Random(case["ragged"])
    counts = [n] * B if n <= 8 else [n] + [r.choice((0, 1, r.randint(1, n))) for _ in range(B - 1)]
    return [L] + [max(c, _log(r, max(1, L // 16), L)) for c in counts[1:]], counts


# ----------------------------------------------------------------- the plain forms (32 bits)
def _rotate(x):
    """Per 32-block along the last axis: the normalised 32-point Walsh-Hadamard transform, stages 1, 2, 4, 8, 16."""
    shape = x.shape
    for h in (1, 2, 4, 8, 16):
        a, b = x.reshape(*shape[:-1], -1, 2, h).unbind(-2)
        x = torch.stack((a + b, a - b), -2)
    return x.reshape(shape) * C_H32


def _rope(x, pos, freqs, interleaved):
    """x [T][H][D], angles in 64 bits."""
    turn = pos.double()[:, None] * freqs
    c, s = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
    y = x.unflatten(-1, (-1, 2)) if interleaved else x.unflatten(-1, (2, -1)).transpose(-1, -2)
    y = torch.stack((y[..., 0] * c - y[..., 1] * s, y[..., 1] * c + y[..., 0] * s), -1)
    return (y if interleaved else y.transpose(-1, -2)).flatten(-2)


def _pow2(e):
    """2^e of whole e in -126 .. 127, exact (a power function need not be)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least E with amax <= 127 * 2^E, in LOW .. TOP."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [.5, 1); 127 = (127 / 128) * 2^7
    return torch.where(amax > 0, e - 7 + (m > 127 / 128), torch.full_like(e, LOW)).clamp(LOW, TOP)


def _codes(y, e):
    return torch.round(y * _pow2(-e)).clamp(-127, 127)


def _values(cache, table):
    """What the pages of table [B][P] hold, K and V [B][tokens][H][D]."""
    c, s, page = cache
    v = c[table].float().unflatten(-2, (-1, TOKENS)) * _pow2(s[table].int() - 127)[..., None, None]
    v = v.flatten(-3, -2).permute(3, 0, 1, 4, 2, 5).flatten(2, 3)  # [2][B][P * page][H][D]
    return v[0], v[1]


def _append_plain(s):
    codes, scales, page = s["cache"]
    q = _rope(s["q"].float(), s["pos"], s["freqs"], s["interleaved"])
    k = _rope(s["k"].float(), s["pos"], s["freqs"], s["interleaved"])
    kv = torch.stack((k, s["v"].float()), 2)  # [T][H][2][D]
    kv = _rotate(kv) if s["rotate"] else kv
    # the touched blocks: what they held before the first new token, then the new rows
    at, first = s["blocks"], s["first"]  # page and block of each; rows that stood in it before
    old = codes.unflatten(-2, (-1, TOKENS))[at[:, 0], :, :, at[:, 1]].float()  # [n][H][2][16][D]
    e_old = torch.where(first[:, None, None] > 0, scales[at[:, 0], :, :, at[:, 1]].int() - 127, LOW)
    new = torch.zeros_like(old)
    new[s["tok_block"], :, :, s["tok_row"]] = kv
    e = torch.maximum(_exponent(new.abs().amax((-1, -2))), e_old)
    row = torch.arange(TOKENS, device=DEV)[:, None]
    keep = (row < first[:, None, None])[:, None, None]
    moved = torch.round(old * _pow2(e_old - e)[..., None, None])
    fresh = (row < s["last"][:, None, None])[:, None, None]
    now = torch.where(keep, moved, torch.where(fresh, _codes(new, e[..., None, None]), old))
    codes.unflatten(-2, (-1, TOKENS))[at[:, 0], :, :, at[:, 1]] = now.to(torch.int8)
    scales[at[:, 0], :, :, at[:, 1]] = (e + 127).to(torch.uint8)
    back = (now * _pow2(e)[..., None, None])[s["read_block"], :, :, s["read_row"]].to(torch.bfloat16)
    return {"q": q.to(s["q_out"].dtype), "k": back[:, :, 0], "v": back[:, :, 1]}


def _attend_plain(s):
    k, v = _values(s["cache"], s["table"])  # [B][L][H][D]
    B, L, H, D = k.shape
    q = s["q"].float()
    q = _rotate(q) if s["rotate"] else q
    n = s["most"]
    rows = torch.zeros(B, n, *q.shape[1:], device=DEV)
    rows[s["tok_seq"], s["tok_row"]] = q
    g = q.shape[1] // H
    rows = rows.unflatten(2, (H, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B][H][g * n][D]
    a = (rows @ k.permute(0, 2, 3, 1)).unflatten(2, (g, n)) * D ** -0.5  # [B][H][g][n][L]
    key = torch.arange(L, device=DEV)
    length = s["lens"].long()[:, None, None]
    pos = (length[:, :, 0] - s["counts"][:, None] + torch.arange(n, device=DEV))[..., None]  # [B][n][1]
    seen = key < length
    if s["causal"]:
        seen = seen & (key <= pos)
    if s["window"]:
        seen = seen & (key > pos - s["window"])
    a.masked_fill_(~seen[:, None, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.transpose(1, 2)).unflatten(2, (g, n)) / torch.where(total > 0, total, torch.ones_like(total))
    o = _rotate(o) if s["rotate"] else o
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["tok_seq"], s["tok_row"]].to(torch.bfloat16)


def _mx_values(codes, scales):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).long()]
    return (v.reshape(codes.shape[0], -1, BLOCK) * _pow2(scales.int() - 127)[..., None]).reshape(codes.shape[0], -1)


def _activate(y, act):
    if act == "relu":
        return y * (y > 0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    return y


def _product_plain(s):
    y = _mx_values(s["ac"], s["asc"]) @ _mx_values(s["wc"], s["ws"]).T
    y = _activate(y if s["bias"] is None else y + s["bias"], s["act"])
    return (y if s["residual"] is None else y + s["residual"].float()).to(s["out"])


# ----------------------------------------------------------------- inputs
def _loud(gen, shape):
    """Activations: N(0, 1) with 1% of the channels twenty times larger."""
    x = torch.randn(*shape, device=DEV, generator=gen)
    n = shape[-1]
    x[..., torch.randperm(n, device=DEV, generator=gen)[: max(1, n // 100)]] *= 20
    return x


def _mx_pack(y):
    """Packed codes [rows][K/2] (element 2i in the low nibble of byte i) and scale bytes [rows][K/32] of rows y."""
    b = y.reshape(y.shape[0], -1, BLOCK)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3).clamp(-127, 127)
    m = b * _pow2(-e)
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    code = (torch.bucketize(m.abs(), steps) + 8 * torch.signbit(m)).reshape(y.shape[0], -1, 2).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _flat(lists):
    return torch.tensor([v for one in lists for v in one], device=DEV)


def _cache(case, gen, lens):
    """Pages in a random order, filled with keys and values of a few widths, and the sequences' tables."""
    B, H, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    per = (max(lens) + page - 1) // page
    x = torch.randn(B * per, H, 2, page, D, device=DEV, generator=gen)
    x *= torch.exp(0.5 * torch.randn(B * per, H, 2, page, 1, device=DEV, generator=gen))
    b = x.unflatten(-2, (-1, TOKENS))
    e = _exponent(b.abs().amax((-1, -2)))
    codes = _codes(b, e[..., None, None]).flatten(-3, -2).to(torch.int8)
    table = torch.randperm(B * per, device=DEV, generator=gen).reshape(B, per).to(torch.int32)
    return codes, (e + 127).to(torch.uint8), table


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(DEV).manual_seed(seed)
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        wc, ws = _mx_pack(torch.randn(N, K, device=DEV, generator=gen) * 0.02)
        ac, asc = _mx_pack(_rotate(_loud(gen, (M, K))))
        s = {"op": op, "act": case["act"], "out": DTYPES[case["out"]],
             "bias": torch.randn(N, device=DEV, generator=gen) if case["bias"] else None,
             "residual": (2 * torch.randn(M, N, device=DEV, generator=gen)).to(DTYPES[case["residual"]])
             if case["residual"] != "none" else None}
        if own:  # the operands as the package keeps them: laid out once
            import hadamard_rotated_w4a4_gb300 as w4
            return dict(s, w=w4.mxfp4_import(wc, ws, rotated=True), a=w4.mxfp4_import(ac, asc, rotated=True))
        return dict(s, wc=wc, ws=ws, ac=ac, asc=asc)
    lens, counts = _lengths(case)
    codes, scales, table = _cache(case, gen, lens)
    T, Hq, Hkv, D = sum(counts), case["Hq"], case["Hkv"], case["D"]
    even = len(set(counts)) == 1  # every sequence has as many new tokens: no offsets are needed
    offsets = [sum(counts[:b]) for b in range(len(counts) + 1)]
    s = {"op": op, "cache": (codes, scales, case["page"]), "table": table, "rotate": case["rotate"],
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "cu": None if even else torch.tensor(offsets, dtype=torch.int32, device=DEV)}
    if own:
        import hadamard_rotated_w4a4_gb300 as w4
        s["cache"] = w4.KvCache8(codes, scales, rotated=case["rotate"])
    if op == "attend":
        q = torch.randn(T, Hq, D, device=DEV, generator=gen) * torch.exp(0.3 * torch.randn(T, Hq, 1, device=DEV, generator=gen))
        s.update(q=q.to(torch.bfloat16), causal=case["causal"], window=case["window"], most=max(counts))
        s["counts"] = torch.tensor(counts, device=DEV)
        s["tok_seq"], s["tok_row"] = _flat([b] * n for b, n in enumerate(counts)), _flat(range(n) for n in counts)
        return s
    # one product's output: q heads, then k, then v
    dtype = DTYPES[case["dtype"]]
    x = _loud(gen, (T, Hq + 2 * Hkv, D)).to(dtype)
    s.update(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], interleaved=case["interleaved"],
             q_out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV),
             freqs=BASE ** (-torch.arange(0, D, 2, dtype=torch.float64, device=DEV) / D))
    before = [L - n for L, n in zip(lens, counts)]
    start = [p // TOKENS * TOKENS for p in before]  # the touched blocks are read back whole
    read = [L - p if n else 0 for L, p, n in zip(lens, start, counts)]
    s["read"] = sum(read)
    s["cu_read"] = torch.tensor([sum(read[:b]) for b in range(len(read) + 1)], dtype=torch.int32, device=DEV)
    if not own:
        per = case["page"] // TOKENS
        blocks = [(b, i) for b in range(len(lens)) if counts[b] for i in range(start[b] // TOKENS, (lens[b] + TOKENS - 1) // TOKENS)]
        at = {x: i for i, x in enumerate(blocks)}
        seq, num = torch.tensor(blocks, device=DEV).unbind(1)
        s["blocks"] = torch.stack((table[seq, num // per].long(), num % per), 1)
        s["first"] = torch.tensor([max(0, before[b] - TOKENS * i) for b, i in blocks], device=DEV)
        s["last"] = torch.tensor([lens[b] - TOKENS * i for b, i in blocks], device=DEV)
        s["pos"] = _flat(range(p, L) for p, L in zip(before, lens))
        s["tok_block"] = _flat([at[b, p // TOKENS] for p in range(before[b], lens[b])] for b in range(len(lens)))
        s["tok_row"] = s["pos"] % TOKENS
        reads = [range(start[b], lens[b]) if counts[b] else () for b in range(len(lens))]
        s["read_block"] = _flat([at[b, p // TOKENS] for p in r] for b, r in enumerate(reads))
        s["read_row"] = _flat(reads) % TOKENS
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import hadamard_rotated_w4a4_gb300 as w4
    if s["op"] == "product":
        return w4.mxfp4_gemm_epilogue(s["w"], s["a"], bias=s["bias"], activation=s["act"], residual=s["residual"], dtype=s["out"])
    if s["op"] == "attend":
        return w4.kv8_attention(s["q"], s["cache"], s["table"], s["lens"], cu=s["cu"], causal=s["causal"], window=s["window"])
    w4.kv8_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], cu=s["cu"], q=s["q"], q_out=s["q_out"],
                  freqs=s["freqs"], interleaved=s["interleaved"])
    k, v = w4.kv8_read(s["cache"], s["table"], s["lens"], s["read"], cu=s["cu_read"], dtype=torch.bfloat16)
    return {"q": s["q_out"], "k": k, "v": v}


def _run_plain(s):
    return {"append": _append_plain, "attend": _attend_plain, "product": _product_plain}[s["op"]](s)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"none": 0, "f32": 4, "bf16": 2}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K // 2 + K // BLOCK) + M * N * (size[case["out"]] + size[case["residual"]]) + 4 * N * case["bias"],
                "flops": 2 * M * N * K}
    lens, counts = _lengths(case)
    T, Hq, Hkv, D = sum(counts), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        read = sum(L - (L - n) // TOKENS * TOKENS for L, n in zip(lens, counts) if n)
        # q, k, v in, q and the codes out, the touched blocks out as bf16
        return {"bytes": T * D * ((Hq + 2 * Hkv) * size[case["dtype"]] + 2 * Hq + 2 * Hkv) + read * 2 * Hkv * D * 2,
                "flops": T * D * (3 * Hq + 14 * Hkv)}
    W = case["window"] or 1 << 40
    if case["causal"]:  # keys that token i of n sees, and keys that a sequence's tokens see together
        pairs = sum(sum(min(L - n + i + 1, W) for i in range(n)) for L, n in zip(lens, counts))
        keys = sum(min(L, W + n - 1) for L, n in zip(lens, counts) if n)
    else:
        pairs, keys = sum(L * n for L, n in zip(lens, counts)), sum(L for L, n in zip(lens, counts) if n)
    return {"bytes": 2 * keys * Hkv * D + 4 * T * Hq * D, "flops": 4 * D * Hq * pairs}


# ----------------------------------------------------------------- the definition in 64 bits
_H = torch.ones(1, 1, dtype=torch.float64)
for _ in range(5):
    _H = torch.cat((torch.cat((_H, _H), 1), torch.cat((_H, -_H), 1)), 0)


def _exact_pow2(e):
    return (e.long() + 1023).bitwise_left_shift(52).view(torch.float64)


def _exact_rotate(y):
    return (y.reshape(-1, BLOCK) @ (_H / math.sqrt(BLOCK)).to(y.device)).reshape(y.shape)


def _exact_rope(x, pos, interleaved):
    T, H, D = x.shape
    j = torch.arange(D // 2, device=x.device)
    z = pos.double()[:, None] * BASE ** (-2.0 * j.double() / D)
    lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + D // 2)
    y = torch.empty_like(x)
    turn = torch.polar(torch.ones_like(z), z)[:, None] * torch.complex(x[..., lo], x[..., hi])
    y[..., lo], y[..., hi] = turn.real, turn.imag
    return y


def _exact_append(case, s, lens, counts):
    codes, scales, page = s["codes"], s["scales"], case["page"]
    qs, ks, vs, t = [], [], [], 0
    for b, (L, n) in enumerate(zip(lens, counts)):
        if n == 0:
            continue
        pos = torch.arange(L - n, L, device=DEV)
        rows = slice(t, t + n)
        t += n
        qs.append(_exact_rope(s["q"][rows].double(), pos, case["interleaved"]))
        new = torch.stack((_exact_rope(s["k"][rows].double(), pos, case["interleaved"]), s["v"][rows].double()), 2)
        new = _exact_rotate(new) if case["rotate"] else new
        lo, hi = (L - n) // TOKENS * TOKENS, (L + TOKENS - 1) // TOKENS * TOKENS
        stood = L - n - lo  # older rows of the first block
        y = torch.zeros(hi - lo, *new.shape[1:], dtype=torch.float64, device=DEV)
        y[stood:stood + n] = new
        y = y.unflatten(0, (-1, TOKENS))
        amax = y.abs().amax((1, 4))  # [blocks][H][2]
        step = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 1e-300)) / 127)).clamp(LOW, TOP)
        if stood:
            pid, blk = int(s["table"][b, lo // page]), lo % page // TOKENS
            was = scales[pid, :, :, blk].double() - 127
            step[0] = torch.maximum(step[0], was)
            old = codes[pid, :, :, blk * TOKENS:blk * TOKENS + stood].double() * _exact_pow2(was)[..., None, None]
            y[0, :stood] = old.permute(2, 0, 1, 3)
        size = _exact_pow2(step)[:, None, :, :, None]
        y = (torch.round(y / size).clamp(-127, 127) * size).flatten(0, 1)[:L - lo]
        ks.append(y[:, :, 0])
        vs.append(y[:, :, 1])
    return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}


def _exact_attend(case, s, lens, counts):
    out, t = [], 0
    g = case["Hq"] // case["Hkv"]
    for b, (L, n) in enumerate(zip(lens, counts)):
        q = s["q"][t:t + n].double()
        t += n
        if n == 0:
            continue
        pids = s["table"][b].long()
        size = _exact_pow2(s["scales"][pids].double() - 127).repeat_interleave(TOKENS, -1)
        kv = (s["codes"][pids].double() * size[..., None]).permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :L]  # [H][2][L][D]
        kv = _exact_rotate(kv) if case["rotate"] else kv
        pos, key = torch.arange(L - n, L, device=DEV)[:, None], torch.arange(L, device=DEV)
        hidden = (key > pos) if case["causal"] else torch.zeros(n, L, dtype=torch.bool, device=DEV)
        if case["window"]:
            hidden = hidden | (key <= pos - case["window"])
        o = torch.empty_like(q)
        for h in range(case["Hq"]):
            w = q[:, h] @ kv[h // g, 0].T / math.sqrt(case["D"])
            o[:, h] = torch.softmax(w.masked_fill(hidden, -math.inf), -1) @ kv[h // g, 1]
        out.append(o)
    return torch.cat(out)


def exact(case, seed):
    global own
    if case["op"] == "product":
        was, own = own, False
        s = prepare(case, seed)
        own = was
        side = []
        for c, e in ((s["ac"], s["asc"]), (s["wc"], s["ws"])):
            code = torch.stack((c % 16, c // 16), -1).reshape(c.shape[0], -1).to(torch.float64)
            m = code % 8
            p, f = torch.floor(m / 2), m % 2  # exponent and mantissa bit
            v = torch.where(p == 0, 0.5 * f, (1 + 0.5 * f) * _exact_pow2(p - 1)) * torch.where(code >= 8, -1.0, 1.0)
            side.append(v * _exact_pow2(e.double() - 127).repeat_interleave(BLOCK, 1))
        y = side[0] @ side[1].T
        y = y if s["bias"] is None else y + s["bias"].double()
        act = case["act"]
        if act == "relu":
            y = y.clamp(min=0)
        elif act == "silu":
            y = y * torch.sigmoid(y)
        elif act == "gelu":
            y = y * 0.5 * torch.erfc(-y / math.sqrt(2))
        elif act == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        return y if s["residual"] is None else y + s["residual"].double()
    was, own = own, False
    s = prepare(case, seed)
    own = was
    s["codes"], s["scales"], _ = s["cache"]
    lens, counts = _lengths(case)
    return (_exact_append if case["op"] == "append" else _exact_attend)(case, s, lens, counts)
