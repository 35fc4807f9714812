"""Refusals of the kv8 calls and of the product with an epilogue: each fails before anything is launched."""
import copy
import ctypes
import pickle

import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from hadamard_rotated_w4a4_gb300 import _Act4Desc, _Epilogue, _Kv8Attn, _Kv8Desc, _Kv8New, _Kv8Seqs

FAKE = 0x10000  # aligned, never dereferenced
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return w4.load_library(build_if_missing=True)


def cache(codes=FAKE, scales=FAKE, pages=8, heads=4, page=64, dim=128, tag=w4.TAG_KV8 | 1):
    return _Kv8Desc(codes, scales, pages, heads, page, dim, tag)


def seqs(table=FAKE, lens=FAKE, cu=None, batch=2, width=4, ldt=4, tokens=6):
    return _Kv8Seqs(table, lens, cu, batch, width, ldt, tokens)


def new(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, freqs=FAKE, ldk=512, ldkh=128, ldv=512, ldvh=128, ldq=1024, ldqh=128, ldo=1024,
        ldoh=128, q_heads=8, nf=64, interleaved=0, x=0, o=0):
    return _Kv8New(k, v, q, q_out, freqs, ldk, ldkh, ldv, ldvh, ldq, ldqh, ldo, ldoh, q_heads, nf, interleaved, x, o)


def attn(q=FAKE, out=2 * FAKE, ldq=1024, ldqh=128, ldo=1024, ldoh=128, q_heads=8, qd=0, od=0, causal=1, window=0, scale=0.1):
    return _Kv8Attn(q, out, ldq, ldqh, ldo, ldoh, q_heads, qd, od, causal, window, scale)


def call(lib, fn, c, s, x=None, *rest):
    ref = lambda d: None if d is None else ctypes.addressof(d)  # noqa: E731
    st = getattr(lib, fn)(ref(c), ref(s), *([] if x is None else [ref(x)]), *rest)
    return w4.STATUS[st], lib.w4a4_last_error().decode()


BAD_CACHE = [
    (dict(tag=w4.TAG_ACT8), "INVALID_ARG"), (dict(page=48), "INVALID_ARG"), (dict(page=256), "INVALID_ARG"),
    (dict(dim=96), "UNSUPPORTED"), (dict(dim=0), "UNSUPPORTED"), (dict(heads=0), "INVALID_ARG"), (dict(heads=-1), "INVALID_ARG"),
    (dict(pages=-1), "INVALID_ARG"), (dict(pages=1 << 31), "INVALID_ARG"), (dict(codes=None), "INVALID_ARG"),
    (dict(scales=None), "INVALID_ARG"), (dict(codes=FAKE + 8), "ALIGNMENT"),
]
BAD_SEQS = [
    (dict(batch=-1), "INVALID_ARG"), (dict(tokens=-1), "INVALID_ARG"), (dict(tokens=1 << 31), "INVALID_ARG"),
    (dict(tokens=7), "INVALID_ARG"), (dict(batch=0), "INVALID_ARG"), (dict(batch=0, cu=FAKE), "INVALID_ARG"), (dict(width=1 << 26, ldt=1 << 26), "INVALID_ARG"),
    (dict(ldt=3), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"),
    (dict(lens=FAKE + 2), "ALIGNMENT"), (dict(table=FAKE + 1), "ALIGNMENT"), (dict(cu=FAKE + 2), "ALIGNMENT"),
]


@pytest.mark.parametrize("fn", ["kv8_append", "kv8_read", "kv8_attention"])
def test_bad_caches_and_sequences(lib, fn):
    args = {"kv8_append": (new(), None), "kv8_read": (None, FAKE, FAKE, 0, 512, 128, 512, 128, None), "kv8_attention": (attn(), None, 0, None)}[fn]
    for kw, want in BAD_CACHE:
        assert call(lib, fn, cache(**kw), seqs(), *args)[0] == "W4A4_ERR_" + want, kw
    for kw, want in BAD_SEQS:
        assert call(lib, fn, cache(), seqs(**kw), *args)[0] == "W4A4_ERR_" + want, kw
    assert call(lib, fn, None, seqs(), *args)[0] == "W4A4_ERR_INVALID_ARG"
    assert call(lib, fn, cache(), None, *args)[0] == "W4A4_ERR_INVALID_ARG"


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(q_out=None), "INVALID_ARG"),
    (dict(q_heads=0), "INVALID_ARG"), (dict(q_heads=-1), "INVALID_ARG"), (dict(freqs=None), "INVALID_ARG"), (dict(freqs=FAKE + 4), "ALIGNMENT"),
    (dict(nf=-8), "INVALID_ARG"), (dict(nf=72), "INVALID_ARG"), (dict(nf=60), "UNSUPPORTED"), (dict(interleaved=2), "INVALID_ARG"),
    (dict(x=2), "INVALID_ARG"), (dict(o=5), "INVALID_ARG"), (dict(ldk=100), "INVALID_ARG"), (dict(ldvh=64), "INVALID_ARG"),
    (dict(ldk=516), "ALIGNMENT"), (dict(ldqh=132), "ALIGNMENT"), (dict(k=FAKE + 8), "ALIGNMENT"), (dict(o=1), "INVALID_ARG"),
    (dict(ldo=2048), "INVALID_ARG"),
])
def test_append_refusals(lib, kw, want):
    assert call(lib, "kv8_append", cache(), seqs(), new(**kw), None)[0] == "W4A4_ERR_" + want


def test_append_without_tokens_or_with_a_null(lib):
    assert call(lib, "kv8_append", cache(), seqs(tokens=0), new(k=None, v=None, q=None, q_out=None, q_heads=0, nf=0, freqs=None), None)[0] == "W4A4_OK"
    assert w4.STATUS[lib.kv8_append(ctypes.addressof(cache()), ctypes.addressof(seqs()), None, None)] == "W4A4_ERR_INVALID_ARG"


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(q_heads=0), "INVALID_ARG"), (dict(q_heads=6), "INVALID_ARG"),
    (dict(causal=2), "INVALID_ARG"), (dict(window=-1), "INVALID_ARG"), (dict(causal=0, window=4), "INVALID_ARG"),
    (dict(scale=NAN), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"), (dict(qd=3), "INVALID_ARG"), (dict(od=-1), "INVALID_ARG"),
    (dict(out=FAKE, od=1), "INVALID_ARG"), (dict(out=FAKE, ldo=2048), "INVALID_ARG"), (dict(ldq=1020), "ALIGNMENT"), (dict(out=FAKE + 4), "ALIGNMENT"),
])
def test_attention_refusals(lib, kw, want):
    assert call(lib, "kv8_attention", cache(), seqs(), attn(**kw), None, 0, None)[0] == "W4A4_ERR_" + want


def test_attention_workspace_and_sizes(lib):
    assert call(lib, "kv8_attention", cache(), seqs(), attn(), FAKE, 1 << 20, None)[0] == "W4A4_ERR_WORKSPACE"
    assert call(lib, "kv8_attention", cache(), seqs(), attn(), FAKE + 4, 1 << 30, None)[0] == "W4A4_ERR_ALIGNMENT"
    assert call(lib, "kv8_attention", cache(), seqs(batch=2049, tokens=2049), attn(), None, 0, None)[0] == "W4A4_ERR_UNSUPPORTED"
    assert call(lib, "kv8_attention", cache(), seqs(batch=1, tokens=(1 << 31) - 256), attn(), None, 0, None)[0] == "W4A4_ERR_UNSUPPORTED"
    assert call(lib, "kv8_attention", cache(), seqs(tokens=0), attn(), None, 0, None)[0] == "W4A4_OK"
    assert lib.kv8_attention_workspace_bytes(128) > 1 << 20 and lib.kv8_attention_workspace_bytes(100) == 0
    assert w4.kv8_attention_workspace_bytes(256) > w4.kv8_attention_workspace_bytes(64)


def mx(rows=64, K=256, rotated=True, tag=None):
    return _Act4Desc(FAKE, FAKE, rows, K, tag if tag is not None else (w4.TAG_MXFP4 | (1 if rotated else 0)))


@pytest.mark.parametrize("kw,want", [
    (dict(act=-1), "INVALID_ARG"), (dict(act=5), "INVALID_ARG"), (dict(bias=FAKE + 2), "ALIGNMENT"), (dict(r=FAKE + 1), "ALIGNMENT"),
    (dict(rd=7), "INVALID_ARG"), (dict(ldr=63), "INVALID_ARG"), (dict(r=4 * FAKE, rd=0), "INVALID_ARG"), (dict(r=4 * FAKE, rd=1, ldr=128), "INVALID_ARG"),
    (dict(y=None), "INVALID_ARG"), (dict(ldy=32), "INVALID_ARG"), (dict(w=mx(K=512)), "MISMATCH"), (dict(w=mx(rotated=False)), "MISMATCH"),
    (dict(yd=2), "INVALID_ARG"),
])
def test_epilogue_refusals(lib, kw, want):
    d = {"bias": FAKE, "r": 2 * FAKE, "ldr": 64, "rd": 0, "act": 0, "y": 4 * FAKE, "yd": 1, "ldy": 64, "w": mx(), **kw}
    e = _Epilogue(d["bias"], d["r"], d["ldr"], d["rd"], d["act"])
    st = lib.mxfp4_gemm_epilogue(ctypes.addressof(d["w"]), ctypes.addressof(mx()), ctypes.addressof(e), d["y"], d["yd"], d["ldy"], None, 0, None)
    assert w4.STATUS[st] == "W4A4_ERR_" + want


def test_epilogue_null(lib):
    assert w4.STATUS[lib.mxfp4_gemm_epilogue(ctypes.addressof(mx()), ctypes.addressof(mx()), None, FAKE, 1, 64, None, 0, None)] == "W4A4_ERR_INVALID_ARG"


def host_cache(pages=4, heads=2, page=32, dim=64, **kw):
    return w4.KvCache8(torch.zeros(pages, heads, 2, page, dim, dtype=torch.int8), torch.zeros(pages, heads, 2, page // 16, dtype=torch.uint8), **kw)


def test_cache_object():
    c = host_cache(rotated=False)
    assert (c.pages, c.heads, c.page, c.dim, c.rotated, c.tag) == (4, 2, 32, 64, False, w4.TAG_KV8)
    for d in (copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert d.codes.data_ptr() != c.codes.data_ptr() and d.desc().codes == d.codes.data_ptr() and not d.rotated
    with pytest.raises(AttributeError):
        c.codes = c.codes
    z = torch.zeros
    for codes, scales, err in (
            (z(4, 2, 2, 32, 64), z(4, 2, 2, 2, dtype=torch.uint8), ValueError),
            (z(4, 2, 3, 32, 64, dtype=torch.int8), z(4, 2, 3, 2, dtype=torch.uint8), ValueError),
            (z(4, 2, 2, 32, 128, dtype=torch.int8)[..., ::2], z(4, 2, 2, 2, dtype=torch.uint8), ValueError),
            (z(4, 2, 2, 32, 64, dtype=torch.int8), z(4, 2, 2, 1, dtype=torch.uint8), ValueError),
            (z(4, 2, 2, 32, 64, dtype=torch.int8), z(4, 2, 2, 2), ValueError),
            (z(4, 2, 2, 24, 64, dtype=torch.int8), z(4, 2, 2, 1, dtype=torch.uint8), w4.W4A4Error),
            (z(4, 2, 2, 32, 96, dtype=torch.int8), z(4, 2, 2, 2, dtype=torch.uint8), w4.W4A4Error)):
        with pytest.raises(err):
            w4.KvCache8(codes, scales)


def test_host_tensors_are_refused():
    c, i = host_cache(), torch.zeros(1, 2, dtype=torch.int32)
    x = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        w4.kv8_append(c, x, x, i, i[0, :1])
    with pytest.raises(ValueError, match="GPU"):
        w4.kv8_attention(x, c, i, i[0, :1])
    with pytest.raises(ValueError, match="GPU"):
        w4.kv8_read(c, i, i[0, :1], 1)
    with pytest.raises(ValueError, match="KvCache8"):
        w4.kv8_read(x, i, i[0, :1], 1)


def test_rope_freqs():
    f = w4.rope_freqs(64, 1e4, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1 and abs(float(f[16]) - 1e-2) < 1e-15


def test_packed_structures_are_the_c_ones():
    """The bytes that the binding passes, against ctypes' layout of the same fields."""
    for pack, kind, values in ((w4._pack_epilogue, _Epilogue, (1, 2, 3, 4, 5)), (w4._pack_kv8_seqs, _Kv8Seqs, range(1, 8)),
                               (w4._pack_kv8_new, _Kv8New, range(1, 19)), (w4._pack_kv8_attn, _Kv8Attn, (*range(1, 12), 0.5))):
        c = kind(*values)
        b = pack(*values)
        assert b == bytes(c)[: len(b)]
        assert len(b) >= max(getattr(kind, n).offset + getattr(kind, n).size for n, _ in kind._fields_)


def test_host_shapes_are_refused():
    c, i = host_cache(), torch.zeros(1, 2, dtype=torch.int32)
    for bad in (torch.zeros(64), torch.zeros(1, 64), torch.zeros(1, 2, 2, 64)):
        with pytest.raises(ValueError):
            w4.kv8_attention(bad, c, i, i[0, :1])
        with pytest.raises(ValueError):
            w4.kv8_append(c, bad, bad, i, i[0, :1])
