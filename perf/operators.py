"""Measured cases of the MXFP4 operators and of the fused norm / SwiGLU quantisers.

``run`` computes each operator either with elementary torch operations in 32 bits
(``own`` false) or with the package's entry points (``own`` true):

* ``quantize``: rotate rows per 32-block, round them to MXFP4, read them back;
* ``product``:  MXFP4 weights times MXFP4 activations, fp32 or bf16 output;
* ``norm``:     residual addition, RMS norm, rotation, int8 per 32-block, read back;
* ``swiglu``:   silu(gate) * up, rotation, int8 per 32-block, read back.

Shapes are those of the package's workloads: hidden 5120, FFN 17408, 512- and
1024-token batches, 2048 -> 768 experts, and ragged ones between.
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-6
C_H32 = 0.1767766922712326  # fl32(1 / sqrt 32)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


# ----------------------------------------------------------------- cases
def listed():
    return [
        # one token's hidden state in front of a projection, each decode step
        {"name": "quantize_token", "op": "quantize", "rows": 1, "K": 5120, "dtype": "f32", "rotate": True},
        # a 1024-token micro-batch in front of the FFN down projection
        {"name": "quantize_ffn", "op": "quantize", "rows": 1024, "K": 17408, "dtype": "f32", "rotate": True},
        # one token through an attention projection
        {"name": "product_token", "op": "product", "M": 1, "K": 5120, "N": 5120, "out": "f32"},
        # a ragged prompt tail through a narrow projection, K an odd number of blocks
        {"name": "product_ragged", "op": "product", "M": 77, "K": 736, "N": 1000, "out": "bf16"},
        # a 512-token micro-batch through an attention projection
        {"name": "product_attn", "op": "product", "M": 512, "K": 5120, "N": 5120, "out": "f32"},
        # a 1024-token micro-batch through the FFN down projection
        {"name": "product_down", "op": "product", "M": 1024, "K": 17408, "N": 5120, "out": "bf16"},
        # a long prompt in one pass through the FFN gate/up projection
        {"name": "product_prompt", "op": "product", "M": 4096, "K": 5120, "N": 17408, "out": "bf16"},
        # one token's residual stream in front of a layer
        {"name": "norm_token", "op": "norm", "M": 1, "K": 5120, "dtype": "bf16", "rotate": True},
        # a 1024-token micro-batch, fp32 product output added to the residual
        {"name": "norm_batch", "op": "norm", "M": 1024, "K": 5120, "dtype": "f32", "rotate": True},
        # a long prompt's residual stream, bf16
        {"name": "norm_prompt", "op": "norm", "M": 16384, "K": 5120, "dtype": "bf16", "rotate": True},
        # an odd batch of an expert's gate and up outputs
        {"name": "swiglu_expert", "op": "swiglu", "M": 67, "K": 768, "dtype": "f32", "rotate": True},
        # a 1024-token micro-batch between gate/up and down
        {"name": "swiglu_ffn", "op": "swiglu", "M": 1024, "K": 17408, "dtype": "bf16", "rotate": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "norm", "swiglu"))
    # whole multiples of 160 (5120 is one), or an odd number of blocks
    K = rng.choice((160 * _log(rng, 1, 108), BLOCK * (2 * _log(rng, 1, 271) + 1)))
    if op == "product":
        N = _log(rng, 64, 17408)
        M = _log(rng, 1, max(1, min(4096, 4096 * 5120 * 17408 // (N * K))))
        return {"op": op, "M": M, "K": K, "N": N, "out": rng.choice(("f32", "bf16"))}
    dtype, rotate = rng.choice(("f32", "bf16")), rng.random() < 0.75
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, min(16384, 1024 * 17408 // K)), "K": K, "dtype": dtype, "rotate": rotate}
    most = 16384 * 5120 if op == "norm" else 1024 * 17408
    return {"op": op, "M": _log(rng, 1, min(16384, most // K)), "K": K, "dtype": dtype, "rotate": rotate}


# ----------------------------------------------------------------- the plain forms (32 bits)
def _rotate(x):
    """Per 32-block along the last axis: the normalised 32-point Walsh-Hadamard transform, stages 1, 2, 4, 8, 16."""
    shape = x.shape
    y = x.reshape(-1, BLOCK)
    h = 1
    while h < BLOCK:
        y = y.reshape(-1, BLOCK // (2 * h), 2, h)
        a, b = y[:, :, 0], y[:, :, 1]
        y = torch.stack((a + b, a - b), 2)
        h *= 2
    return (y.reshape(shape) * C_H32) if x.dtype == torch.float32 else y.reshape(shape) / math.sqrt(BLOCK)


def _mx_round(y):
    """MXFP4 of rows y: e2m1 values (fp) and block exponents, the values read back being values * 2^exponent."""
    b = y.reshape(*y.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)  # floor(log2 amax) - 2
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = torch.ldexp(b, -e)
    m = v.abs()
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; halfway cases go to the even code
    q = (0.5 * (m > 0.25) + 0.5 * (m >= 0.75) + 0.5 * (m > 1.25) + 0.5 * (m >= 1.75)
         + 1.0 * (m > 2.5) + 1.0 * (m >= 3.5) + 2.0 * (m > 5.0)).to(y.dtype)
    return torch.copysign(q, v), e


def _mx_pack(y):
    """Packed codes [rows][K/2] (element 2i in the low nibble of byte i) and scale bytes [rows][K/32] of rows y."""
    q, e = _mx_round(y)
    steps = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    code = torch.bucketize(q.abs().float(), steps) + 8 * torch.signbit(q)
    code = code.reshape(y.shape[0], -1, 2).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _mx_values(codes, scales, dtype):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).long()]
    s = torch.exp2(scales.to(dtype) - 127)
    return (v.reshape(codes.shape[0], -1, BLOCK) * s[..., None]).reshape(codes.shape[0], -1)


def _int8_back(y):
    """int8 per 32-block (scale amax / 127, round half away from zero), read back."""
    b = y.reshape(y.shape[0], -1, BLOCK)
    d = b.abs().amax(-1, keepdim=True) / 127
    v = b * torch.where(d == 0, torch.zeros_like(d), 1 / d)
    q = torch.trunc(v)
    q = (q + torch.copysign(((v - q).abs() >= 0.5).to(v.dtype), v)).clamp(-127, 127)
    return (q * d).reshape(y.shape)


def _norm(x, r, g):
    h = x + r
    return h, h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * g


# ----------------------------------------------------------------- inputs
def _rows(gen, rows, K, dtype):
    """Activations: N(0, 1) with 1% of the channels twenty times larger."""
    x = torch.randn(rows, K, device=DEV, generator=gen)
    loud = torch.randperm(K, device=DEV, generator=gen)[: max(1, K // 100)]
    x[:, loud] *= 20
    return x.to(dtype)


def _product_inputs(case, seed):
    """Weight and activation codes and scales: N(0, 0.02) weights and loud-channel activations, rotated, in MXFP4."""
    gen = torch.Generator(DEV).manual_seed(seed)
    w = torch.randn(case["N"], case["K"], device=DEV, generator=gen) * 0.02
    x = _rows(gen, case["M"], case["K"], torch.float32)
    return _mx_pack(_rotate(w)) + _mx_pack(_rotate(x))


def prepare(case, seed):
    op = case["op"]
    if op == "product":
        wc, ws, ac, asc = _product_inputs(case, seed)
        s = {"out": DTYPES[case["out"]]}
        if own:  # the operands as the package keeps them: laid out once
            import hadamard_rotated_w4a4_gb300 as w4
            return dict(s, op=op, w=w4.mxfp4_import(wc, ws, rotated=True), a=w4.mxfp4_import(ac, asc, rotated=True))
        return dict(s, op=op, wc=wc, ws=ws, ac=ac, asc=asc)
    gen = torch.Generator(DEV).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"op": op, "rotate": case["rotate"]}
    if op == "quantize":
        return dict(s, x=_rows(gen, case["rows"], case["K"], dtype))
    M, K = case["M"], case["K"]
    if op == "norm":
        x = _rows(gen, M, K, dtype)
        r = (torch.randn(M, K, device=DEV, generator=gen) * 2).to(torch.bfloat16)  # the residual stream
        g = 1 + 0.1 * torch.randn(K, device=DEV, generator=gen)
        return dict(s, x=x, r=r, g=g, h=torch.empty_like(r))
    gu = torch.randn(M, 2 * K, device=DEV, generator=gen).to(dtype)  # one product's output: gate, then up
    return dict(s, gate=gu[:, :K], up=gu[:, K:])


# ----------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import hadamard_rotated_w4a4_gb300 as w4
    op = s["op"]
    if op == "quantize":
        return w4.mxfp4_dequantize(w4.mxfp4_rotate_quantize(s["x"], rotate=s["rotate"]))
    if op == "product":
        return w4.mxfp4_gemm(s["w"], s["a"], dtype=s["out"])
    if op == "norm":
        a = w4.w4a8_rmsnorm_quantize_act(s["x"], s["g"], eps=EPS, residual=s["r"], residual_out=s["h"], rotate=s["rotate"])
        return {"residual": s["h"], "values": w4.w4a8_dequantize_act(a, dtype=torch.bfloat16)}
    a = w4.w4a8_swiglu_quantize_act(s["gate"], s["up"], rotate=s["rotate"])
    return w4.w4a8_dequantize_act(a, dtype=torch.bfloat16)


def _run_plain(s):
    op = s["op"]
    if op == "product":
        return (_mx_values(s["ac"], s["asc"], torch.float32) @ _mx_values(s["wc"], s["ws"], torch.float32).T).to(s["out"])
    if op == "quantize":
        x = s["x"].float()
        q, e = _mx_round(_rotate(x) if s["rotate"] else x)
        return torch.ldexp(q, e).reshape(x.shape)
    if op == "norm":
        h, y = _norm(s["x"].float(), s["r"].float(), s["g"])
        return {"residual": h.to(s["r"].dtype), "values": _int8_back(_rotate(y) if s["rotate"] else y).to(torch.bfloat16)}
    g, u = s["gate"].float(), s["up"].float()
    y = g / (1 + torch.exp(-g)) * u
    return _int8_back(_rotate(y) if s["rotate"] else y).to(torch.bfloat16)


# ----------------------------------------------------------------- what a pass cannot do without
def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op, K = case["op"], case["K"]
    if op == "product":
        M, N = case["M"], case["N"]
        return {"bytes": (M + N) * (K // 2 + K // BLOCK) + M * N * _size(case["out"]), "flops": 2 * M * N * K}
    if op == "quantize":
        return {"bytes": case["rows"] * K * (_size(case["dtype"]) + 4), "flops": case["rows"] * K * 10}
    n = case["M"] * K
    if op == "norm":
        return {"bytes": n * (_size(case["dtype"]) + 2 + 2 + 2) + 4 * K, "flops": n * 14}
    return {"bytes": n * (2 * _size(case["dtype"]) + 2), "flops": n * 14}


# ----------------------------------------------------------------- the definition in 64 bits
_H = torch.ones(1, 1, dtype=torch.float64)
for _ in range(5):
    _H = torch.cat((torch.cat((_H, _H), 1), torch.cat((_H, -_H), 1)), 0)


def _exact_rotate(y):
    return (y.reshape(-1, BLOCK) @ (_H / math.sqrt(BLOCK)).to(y.device)).reshape(y.shape)


def _exact_int8(y):
    b = y.reshape(-1, BLOCK)
    d = b.abs().amax(1, keepdim=True) / 127
    q = torch.where(d > 0, b / d, torch.zeros_like(b))
    return (torch.sign(q) * torch.floor(q.abs() + 0.5) * d).reshape(y.shape)


def exact(case, seed):
    op = case["op"]
    if op == "product":
        wc, ws, ac, asc = _product_inputs(case, seed)
        side = []
        for c, s in ((ac, asc), (wc, ws)):
            code = torch.stack((c % 16, c // 16), -1).reshape(c.shape[0], -1).to(torch.float64)
            m = code % 8
            p, f = torch.floor(m / 2), m % 2  # exponent and mantissa bit
            v = torch.where(p == 0, 0.5 * f, (1 + 0.5 * f) * 2.0 ** (p - 1)) * torch.where(code >= 8, -1.0, 1.0)
            side.append(v * (2.0 ** (s.to(torch.float64) - 127)).repeat_interleave(BLOCK, 1))
        return side[0] @ side[1].T
    s = prepare(case, seed)
    if op == "quantize":
        y = s["x"].double()
        y = _exact_rotate(y) if s["rotate"] else y
        b = y.reshape(-1, BLOCK)
        a = b.abs().amax(1, keepdim=True)
        scale = 2.0 ** (torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))) - 2)
        v = b / scale
        grid = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
        at = torch.bucketize(v.abs(), (grid[1:] + grid[:-1]) / 2)
        return (torch.sign(v) * grid[at] * scale).reshape(y.shape)
    if op == "norm":
        h = s["x"].double() + s["r"].double()
        y = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["K"] + EPS) * s["g"].double()
        return {"residual": h, "values": _exact_int8(_exact_rotate(y) if s["rotate"] else y)}
    g, u = s["gate"].double(), s["up"].double()
    y = torch.sigmoid(g) * g * u
    return _exact_int8(_exact_rotate(y) if s["rotate"] else y)
