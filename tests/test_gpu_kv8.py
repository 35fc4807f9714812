"""The 8-bit paged keys and values on the GPU: appending against the oracle, bit for bit where no angle is involved,
else within the fp32 error of the angles; reading back; attention against 64 bits (kv8_testutil)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
import oracle
from kv8_testutil import U, check_attention, ints, make_cache, make_table, values
from w4a4_testutil import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def offsets(counts):
    return [0] + list(np.cumsum(counts))


def rows(rng, T, H, D, dtype, dev):
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x[..., rng.integers(0, D, max(1, D // 64))] *= 20
    return torch.from_numpy(x).to(dev).to(dtype)


# ----------------------------------------------------------------- append and read
@pytest.mark.parametrize("dim,page,dtype", [(64, 16, torch.float32), (128, 64, torch.bfloat16), (256, 32, torch.bfloat16),
                                            (128, 128, torch.float32), (64, 32, torch.bfloat16), (256, 16, torch.float32)])
@pytest.mark.parametrize("rotated", [False, True])
def test_append_in_pieces_is_the_oracles(dev, dim, page, dtype, rotated):
    """Pieces of many lengths into the same sequences, empty ones among them: codes and scales equal after each."""
    rng = np.random.default_rng(dim + page)
    H, B = 3, 4
    lens, pages = [0] * B, 40
    table, t = make_table(rng, dev, pages, [150] * B, page, 150 // page + 2)
    cache = w4.alloc_kv8(pages, H, dim, page, dev, rotated)
    codes, scales = cache.codes.cpu().numpy().copy(), cache.scales.cpu().numpy().copy()
    for step, counts in enumerate(([1, 5, 0, 17], [1, 1, 1, 1], [30, 0, 2, 16], [15, 15, 15, 15], [1, 64, 33, 3])):
        T = sum(counts)
        x = rows(rng, T, 2 * H, dim, dtype, dev) * (1.0 + 3 * step)  # scales that grow
        k, v = x[:, :H], x[:, H:]
        lens = [L + n for L, n in zip(lens, counts)]
        even = len(set(counts)) == 1
        w4.kv8_append(cache, k, v, t, ints(lens, dev), cu=None if even else ints(offsets(counts), dev))
        f = x.float().cpu().numpy()
        f = oracle.rotate_h32(f) if rotated else f
        oracle.kv8_append(codes, scales, f[:, :H], f[:, H:], table, lens, counts)
        assert np.array_equal(cache.scales.cpu().numpy(), scales)
        assert np.array_equal(cache.codes.cpu().numpy(), codes)
    for want in (torch.float32, torch.bfloat16):
        T = sum(lens)
        k, v = w4.kv8_read(cache, t, ints(lens, dev), T, cu=ints(offsets(lens), dev), dtype=want)
        ref = np.concatenate([values(codes, scales, table[b], L) for b, L in enumerate(lens)], axis=1)
        assert np.array_equal(k.double().cpu().numpy(), ref[0]) and np.array_equal(v.double().cpu().numpy(), ref[1])
    w4.w4a4_check()


@pytest.mark.parametrize("dim,nf,interleaved", [(64, 32, False), (128, 64, False), (256, 128, False), (128, 64, True),
                                                (128, 24, False), (256, 8, False), (64, 5, True), (256, 128, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_positions(dev, dim, nf, interleaved, dtype):
    """q, and the keys' codes, at near and far positions.  A cosine: the turn in fp32 half a unit of 1/2, 2 pi 2^-25 of angle,
    and sincospif 2 ulp: 3.2 U + 2 U; a turned value: (|a| + |b|) (5.2 + 1.5) U, 14 U B with B the row's largest magnitude.
    H32: 5.66 (14 + 6) U of sqrt 2 B: 160 U B."""
    rng = np.random.default_rng(nf)
    H, Hq, page, counts = 2, 5, 32, [1, 40, 3]
    lens = [1, 100, 3]
    freqs = w4.rope_freqs(2 * nf, 1e6, dev)
    f = freqs.cpu().numpy()
    for far in (0, 1 << 20):
        shift = far // page
        table, t = make_table(rng, dev, 16, lens, page)
        wide = torch.full((3, shift + t.shape[1]), -1, dtype=torch.int32, device=dev)
        wide[:, shift:] = t
        cache = w4.alloc_kv8(16, H, dim, page, dev, True)
        T = sum(counts)
        x = rows(rng, T, Hq + 2 * H, dim, dtype, dev)
        q_out = torch.empty(T, Hq, dim, dtype=torch.float32, device=dev)
        w4.kv8_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], wide, ints([L + far for L in lens], dev), cu=ints(offsets(counts), dev),
                      q=x[:, :Hq], q_out=q_out, freqs=freqs, interleaved=interleaved)
        pos = np.concatenate([np.arange(L - n, L) + far for L, n in zip(lens, counts)])
        xs = x.double().cpu().numpy()
        B = np.abs(xs).max(axis=-1, keepdims=True)
        want = oracle.rope(xs[:, :Hq], pos, f, interleaved)
        assert (np.abs(q_out.double().cpu().numpy() - want) <= 14 * U * B[:, :Hq]).all()
        back = w4.kv8_read(cache, wide, ints([L + far for L in lens], dev), T, cu=ints(offsets(counts), dev))[0].double().cpu().numpy()
        y = oracle.rotate_h32(oracle.rope(xs[:, Hq:Hq + H], pos, f, interleaved), dtype=np.float64)
        tol = 160 * U * B[:, Hq:Hq + H]
        scales = cache.scales.cpu().numpy().astype(float)
        at = 0
        for b, (L, n) in enumerate(zip(lens, counts)):
            p = np.arange(L - n, L)
            step = 2.0 ** (scales[table[b][p // page], :, 0, p % page // 16] - 127)[..., None]
            lo, hi = np.rint((y[at:at + n] - tol[at:at + n]) / step) * step, np.rint((y[at:at + n] + tol[at:at + n]) / step) * step
            assert (back[at:at + n] >= lo).all() and (back[at:at + n] <= hi).all()
            at += n
        # in place, and as bf16 where that is the type
        q = x[:, :Hq].clone()
        assert w4.kv8_append(cache, x[:, Hq:Hq + H], x[:, Hq + H:], wide, ints([L + far for L in lens], dev), cu=ints(offsets(counts), dev),
                             q=q, freqs=freqs, interleaved=interleaved) is q
        assert torch.equal(q, q_out.to(dtype))
    w4.w4a4_check()


def test_positions_of_any_frequency(dev):
    """Negative, zero and tiny ones, several turns a position, and NaN and infinities, which reach their pairs alone.  An
    angle's own roundings, in 64 bits here and in 2^-64 turns there, are 2^-51 of it at most: 3e-10 at 1000 x 700."""
    rng = np.random.default_rng(18)
    D, L = 64, 1000
    f = np.concatenate([[-1.0, 0.0, -0.0, 700.0, -700.0, 1e-9, -1e-300, 2 * np.pi, np.nan, np.inf, -np.inf, 3.0], rng.standard_normal(20)])
    freqs = torch.from_numpy(f).to(dev)
    x = rows(rng, L, 3, D, torch.float32, dev)
    cache, t = w4.alloc_kv8(63, 1, D, 16, dev), ints(range(63), dev)[None]
    q = w4.kv8_append(cache, x[:, 1:2], x[:, 2:], t, ints([L], dev), q=x[:, :1], q_out=torch.empty_like(x[:, :1]), freqs=freqs)
    q, xs = q.double().cpu().numpy(), x.double().cpu().numpy()[:, :1]
    bad = np.tile(~np.isfinite(f), 2)
    assert np.isnan(q[..., bad]).all() and np.isfinite(q[..., ~bad]).all()
    want = oracle.rope(xs, np.arange(L), np.where(np.isfinite(f), f, 0), False)
    B = np.abs(xs).max(axis=-1, keepdims=True)
    assert (np.abs(q - want) <= (14 * U + 1e-9) * B)[..., ~bad].all()
    assert (cache.scales[:, 0, 0] == 255).all() and (cache.scales[:, 0, 1] != 255).all()
    w4.w4a4_check()


def test_append_strides_and_rows_behind(dev):
    """Views of one product's output, padded rows, and tokens past the last offset: nothing but the named rows is written."""
    rng = np.random.default_rng(1)
    H, Hq, D, page = 2, 4, 128, 16
    lens, counts = [20, 9], [7, 9]
    table, t = make_table(rng, dev, 6, lens, page)
    x = rows(rng, 24, Hq + 2 * H + 3, D, torch.bfloat16, dev)  # 24 rows, 16 of them tokens
    cache, codes, scales = make_cache(rng, dev, 6, H, page, D)
    out = torch.full((24, Hq + 1, D), 7.0, dtype=torch.bfloat16, device=dev)
    w4.kv8_append(cache, x[:, Hq:Hq + H], x[:, Hq + H + 1:Hq + 2 * H + 1], t, ints(lens, dev), cu=ints([0, 7, 16], dev),
                  q=x[:, :Hq], q_out=out[:, 1:], freqs=w4.rope_freqs(D, device=dev))
    assert (out[16:] == 7).all() and (out[:, 0] == 7).all() and not (out[:16, 1:] == 7).all(dim=-1).any()
    f = oracle.rotate_h32(x.float().cpu().numpy())
    ref_k, ref_s = codes.copy(), scales.copy()
    oracle.kv8_append(ref_k, ref_s, f[:, Hq:Hq + H], f[:, Hq + H + 1:Hq + 2 * H + 1], table, lens, counts)
    assert np.array_equal(cache.codes.cpu().numpy()[:, :, 1], ref_k[:, :, 1])  # V: no positions
    assert np.array_equal(cache.scales.cpu().numpy()[:, :, 1], ref_s[:, :, 1])
    new = ref_k != codes  # rows that the oracle left alone are alone
    touched = new.any(axis=(1, 2, 4))
    assert np.array_equal((cache.codes.cpu().numpy() != codes).any(axis=(1, 2, 4)) & ~touched, np.zeros_like(touched))
    k, v = (torch.full((24, H, D), 5.0, device=dev) for _ in range(2))
    w4.kv8_read(cache, t, ints(lens, dev), 24, cu=ints([0, 7, 16], dev), k=k, v=v)
    assert (k[16:] == 5).all() and (v[16:] == 5).all()
    w4.w4a4_check()


def test_append_extremes(dev):
    """Zeros, magnitudes past the scales' range, infinities and NaN."""
    D, page = 64, 16
    for value, want in ((0.0, 0.0), (1e30, 127 * 2.0 ** 40), (-1e30, -127 * 2.0 ** 40), (2.0 ** -60, 0.0), (3.0 * 2.0 ** -40, 3.0 * 2.0 ** -40),
                        (float("nan"), float("nan")), (float("inf"), float("nan"))):
        cache = w4.alloc_kv8(1, 1, D, page, dev, False)
        t, one = ints([0], dev)[None], torch.full((1, 1, D), 1.0, device=dev)
        x = torch.zeros(1, 1, D, device=dev)
        x[0, 0, 3] = value
        w4.kv8_append(cache, x, one, t, ints([1], dev))
        k, v = w4.kv8_read(cache, t, ints([1], dev), 1)
        assert (v == 1).all()
        assert torch.isnan(k).all() if np.isnan(want) else float(k[0, 0, 3]) == want
        w4.kv8_append(cache, one, one, t, ints([2], dev))  # behind it: NaN stays until row 0 is written again
        k, _ = w4.kv8_read(cache, t, ints([2], dev), 2)
        assert torch.isnan(k).all() == np.isnan(want)
        w4.kv8_append(cache, one, one, t, ints([1], dev))
        assert (w4.kv8_read(cache, t, ints([1], dev), 1)[0] == 1).all()
    w4.w4a4_check()


def test_growing_scales_stay_within_a_step(dev):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((16, 1, 64)).astype(np.float32) * np.exp2(np.arange(16))[:, None, None].astype(np.float32)
    cache, t = w4.alloc_kv8(1, 1, 64, 16, dev, True), ints([0], dev)[None]
    k = torch.from_numpy(x).to(dev)
    for i in range(16):
        w4.kv8_append(cache, k[i:i + 1], k[i:i + 1], t, ints([i + 1], dev))
    back = w4.kv8_read(cache, t, ints([16], dev), 16)[0].double().cpu().numpy()
    step = 2.0 ** (float(cache.scales[0, 0, 0, 0]) - 127)
    assert np.abs(back - oracle.rotate_h32(x)).max() < step


def test_pages_lengths_and_offsets_out_of_range(dev):
    """Skipped, flagged, and nothing else touched."""
    rng = np.random.default_rng(2)
    H, D, page = 1, 64, 16
    x = rows(rng, 8, 3, D, torch.float32, dev)
    k, v, q = x[:, :1], x[:, 1:2], x[:, 2:]
    good = ints([1, 2], dev)[None]
    for table, lens, cu in ((ints([1, 4], dev)[None], [20], None), (ints([-1, 2], dev)[None], [8], None), (good, [40], None),
                            (good, [5], None), (good, [-3], None), (good, [20], [0, 9]), (good, [20], [-1, 4]), (good, [20], [6, 2])):
        cache, codes, scales = make_cache(rng, dev, 4, H, page, D)
        cu = None if cu is None else ints(cu, dev)
        for call in (lambda: w4.kv8_append(cache, k, v, table, ints(lens, dev), cu=cu, q=q, q_out=torch.empty_like(q)),
                     lambda: w4.kv8_read(cache, table, ints(lens, dev), 8, cu=cu),
                     lambda: w4.kv8_attention(q, cache, table, ints(lens, dev), cu=cu)):
            w4.w4a4_check()
            call()
            if call.__code__.co_names.count("kv8_attention") and lens == [5]:
                w4.w4a4_check()  # queries before a sequence's start see nothing: no fault
                continue
            with pytest.raises(w4.W4A4Error) as e:
                w4.w4a4_check()
            assert e.value.status_name == "W4A4_ERR_DEVICE_FLAG"
        now = cache.codes.cpu().numpy()
        assert np.array_equal(now[0], codes[0]) and np.array_equal(now[3], codes[3])
    w4.w4a4_check()


# ----------------------------------------------------------------- attention
CASES = [
    # dim, heads, group, page, lens, counts
    (128, 2, 5, 64, [1], [1]), (128, 2, 5, 64, [1000], [1]), (64, 4, 1, 16, [17, 1, 16, 300], [1, 1, 1, 1]),
    (256, 1, 16, 32, [129, 5], [1, 1]), (128, 1, 3, 128, [5000], [1]), (128, 8, 2, 16, [15, 2000, 33], [1, 1, 1]),
    (64, 2, 8, 32, [700, 90], [2, 2]), (256, 2, 5, 16, [260, 8], [3, 3]), (128, 2, 2, 64, [64, 63], [8, 8]),
    (128, 1, 7, 16, [100, 3, 50, 0, 31], [20, 1, 0, 0, 31]), (64, 3, 4, 64, [333], [200]), (256, 1, 2, 128, [300, 290], [100, 1]),
    (128, 2, 1, 32, [513], [513]), (64, 1, 24, 16, [77], [5]), (128, 1, 128, 16, [99, 40], [1, 3]),
    # more new tokens than there are, and no tokens at all
    (128, 2, 3, 16, [10, 50], [30, 50]), (64, 1, 2, 32, [0, 3], [40, 9]), (256, 1, 1, 16, [2, 0], [5, 5]),
]


WIDE = 1 << 19  # keys a table has places for: which kernel takes many rows of few keys goes by this


@pytest.mark.parametrize("dim,heads,group,page,lens,counts", CASES)
@pytest.mark.parametrize("rotated,wide", [(True, False), (False, False), (True, True)])
def test_attention(dev, dim, heads, group, page, lens, counts, rotated, wide):
    rng = np.random.default_rng(dim + sum(lens))
    pages = sum((L + page - 1) // page for L in lens) + 2
    cache, codes, scales = make_cache(rng, dev, pages, heads, page, dim, rotated)
    table, t = make_table(rng, dev, pages, lens, page, WIDE // page if wide else None)
    T, Hq = sum(counts), heads * group
    q = rows(rng, T, Hq, dim, torch.bfloat16, dev) * 0.2
    cu = None if len(set(counts)) == 1 else ints(offsets(counts), dev)
    last = ints(lens, dev)
    for causal, window in ((True, 0), (False, 0), (True, 1), (True, 37)):
        for dtype in (torch.bfloat16, torch.float32):
            got = w4.kv8_attention(q, cache, t, last, cu=cu, causal=causal, window=window, dtype=dtype)
            assert got.dtype == dtype and got.shape == q.shape
            check_attention(got, q, codes, scales, table, lens, counts, causal=causal, window=window, rotated=rotated)
        again = w4.kv8_attention(q, cache, t, last, cu=cu, causal=causal, window=window, dtype=dtype)
        assert torch.equal(got, again)  # fixed order of sums
        alone = w4.kv8_attention(q, cache, t, last, cu=cu, causal=causal, window=window, dtype=dtype, ws=None)
        check_attention(alone, q, codes, scales, table, lens, counts, causal=causal, window=window, rotated=rotated)
    w4.w4a4_check()


@pytest.mark.parametrize("dim,heads,group,page,lens,counts,window", [
    (256, 2, 5, 32, [2500, 700, 130], [8, 8, 8], 0), (128, 2, 4, 64, [3000, 1], [100, 1], 0), (64, 1, 8, 16, [2100, 40, 900], [60, 30, 3], 0),
    (128, 1, 17, 128, [5000], [1], 0), (64, 2, 3, 64, [1800], [700], 300), (256, 1, 20, 16, [1700, 1600], [1, 30], 0)])
def test_attention_of_many_rows_over_many_keys(dev, dim, heads, group, page, lens, counts, window):
    """More key tiles than any ring of the kernel holds, whole and in parts."""
    rng = np.random.default_rng(dim + len(lens))
    pages = sum((L + page - 1) // page for L in lens)
    cache, codes, scales = make_cache(rng, dev, pages, heads, page, dim)
    table, t = make_table(rng, dev, pages, lens, page)
    q = rows(rng, sum(counts), heads * group, dim, torch.bfloat16, dev) * 0.3
    cu = None if len(set(counts)) == 1 else ints(offsets(counts), dev)
    for ws in (True, None):
        got = w4.kv8_attention(q, cache, t, ints(lens, dev), cu=cu, window=window, dtype=torch.float32, ws=ws)
        check_attention(got, q, codes, scales, table, lens, counts, window=window)
        assert torch.equal(got, w4.kv8_attention(q, cache, t, ints(lens, dev), cu=cu, window=window, dtype=torch.float32, ws=ws))
    w4.w4a4_check()


def test_attention_of_many_sequences_of_many_rows(dev):
    """More sequences than a warp's lanes: whole row tiles, and (with one head) tiles cut into parts."""
    rng = np.random.default_rng(14)
    for B, H, g, D, page in ((40, 1, 3, 128, 32), (45, 2, 2, 64, 16)):
        lens = [int(x) for x in rng.integers(30, 900, B)]
        counts = [int(x) for x in rng.integers(0, 30, B)]
        pages = sum((L + page - 1) // page for L in lens)
        cache, codes, scales = make_cache(rng, dev, pages, H, page, D)
        table, t = make_table(rng, dev, pages, lens, page)
        q = rows(rng, sum(counts), H * g, D, torch.bfloat16, dev)
        got = w4.kv8_attention(q, cache, t, ints(lens, dev), cu=ints(offsets(counts), dev))
        check_attention(got, q, codes, scales, table, lens, counts)
    w4.w4a4_check()


def test_attention_gives_up_on_a_bounded_wait(dev):
    """A loader held back longer than the waits' limit: the kernel returns by itself, the check says so, the next call is right."""
    rng = np.random.default_rng(13)
    for dim in (128, 256):
        cache, codes, scales = make_cache(rng, dev, 8, 1, 64, dim)
        table, t = make_table(rng, dev, 8, [400], 64, WIDE // 64)
        q = rows(rng, 50, 2, dim, torch.bfloat16, dev)
        w4.w4a4_debug_set_wait_limit(2_000_000, 20_000_000)
        try:
            w4.kv8_attention(q, cache, t, ints([400], dev))
            with pytest.raises(w4.W4A4Error) as e:
                w4.w4a4_check()
            assert e.value.status_name == "W4A4_ERR_TIMEOUT"
        finally:
            w4.w4a4_debug_set_wait_limit()
        got = w4.kv8_attention(q, cache, t, ints([400], dev))
        w4.w4a4_check()
        check_attention(got, q, codes, scales, table, [400], [50])


def test_attention_types_strides_scale(dev):
    rng = np.random.default_rng(5)
    lens, counts, page, H, g, D = [90, 40], [30, 2], 32, 2, 3, 128
    cache, codes, scales = make_cache(rng, dev, 8, H, page, D)
    for width in (9, WIDE // page):
        table, t = make_table(rng, dev, 8, lens, page, width)
        for o_type in (torch.float32, torch.bfloat16):
            x = rows(rng, 40, H * g + 2, D, o_type, dev) * 0.3
            q = x[:, 1:1 + H * g]
            out = torch.full((40, H * g + 2, D), 3.0, device=dev, dtype=o_type)
            w4.kv8_attention(q, cache, t, ints(lens, dev), cu=ints([0, 30, 32], dev), scale=-0.05, out=out[:, 2:])
            assert (out[:, :2] == 3).all() and (out[32:] == 3).all()
            check_attention(out[:32, 2:], q[:32], codes, scales, table, lens, counts, scale=-0.05)
            y = q.clone()  # in place
            w4.kv8_attention(y, cache, t, ints(lens, dev), cu=ints([0, 30, 32], dev), scale=-0.05, out=y)
            assert torch.equal(y[:32], out[:32, 2:]) and torch.equal(y[32:], q[32:])
    assert w4.kv8_attention(q[:0], cache, t, ints(lens, dev), cu=ints([0, 0, 0], dev)).shape == (0, H * g, D)


def test_attention_of_wide_scales_and_loud_queries(dev):
    """Scales at both ends of their range in one sequence (each V block weighs in the softmax alike), and q of any size."""
    rng = np.random.default_rng(6)
    lens, counts, page, H, g, D = [100], [1], 16, 1, 4, 64
    cache, codes, scales = make_cache(rng, dev, 8, H, page, D, rotated=False)
    scales[:, :, 1] = 127 + rng.integers(-40, 41, scales[:, :, 1].shape)
    scales[:, :, 0] = 127 - 14
    cache.scales.copy_(torch.from_numpy(scales))
    table, t = make_table(rng, dev, 8, lens, page)
    for size in (1.0, 1e-30, 1e6):
        q = rows(rng, 1, g, D, torch.bfloat16, dev) * size
        got = w4.kv8_attention(q, cache, t, ints(lens, dev), scale=0.1 / size, dtype=torch.float32)
        check_attention(got, q, codes, scales, table, lens, counts, scale=0.1 / size, rotated=False)


def test_pages_that_were_only_zeroed_hold_zeros(dev):
    """Blocks that no append wrote, in the middle of a sequence: keys and values of zero, in every kernel alike."""
    D = 128
    cache = w4.alloc_kv8(8, 1, D, 32, dev)
    t = torch.full((1, WIDE // 32), -1, dtype=torch.int32, device=dev)
    t[0, :8] = ints(range(8), dev)
    rng = np.random.default_rng(17)
    x = rows(rng, 40, 2, D, torch.bfloat16, dev)
    w4.kv8_append(cache, x[:, :1], x[:, 1:], t, ints([200], dev))
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    table = t.cpu().numpy()
    k, v = w4.kv8_read(cache, t, ints([200], dev), 200)
    assert (k[:144] == 0).all() and (v[:144] == 0).all() and torch.isfinite(k).all()
    for n, width in ((1, 8), (30, 8), (30, WIDE // 32)):
        q = rows(rng, n, 2, D, torch.bfloat16, dev)
        check_attention(w4.kv8_attention(q, cache, t[:, :width], ints([200], dev), dtype=torch.float32), q, codes, scales, table, [200], [n])


def test_attention_nan_reaches_who_sees_it(dev):
    """A NaN block in places that a row does not see does not touch it; one that it sees makes it NaN."""
    rng = np.random.default_rng(7)
    page, H, g, D, L, n = 16, 1, 2, 64, 100, 70
    table, t = make_table(rng, dev, 8, [L], page, WIDE // page)
    for kind in (0, 1):
        for n, window in ((70, 0), (70, 20), (4, 0), (4, 20)):
            cache, codes, scales = make_cache(rng, dev, 8, H, page, D)
            q = rows(rng, n, H * g, D, torch.bfloat16, dev)
            clean = w4.kv8_attention(q, cache, t, ints([L], dev), window=window)
            cache.scales[int(table[0, 3]), 0, kind, 0] = 255  # keys 48 .. 63
            got = w4.kv8_attention(q, cache, t, ints([L], dev), window=window)
            pos = np.arange(L - n, L)
            sees = (pos >= 48) & ((window == 0) | (pos - window < 63))
            assert torch.isnan(got[torch.from_numpy(sees)]).all()
            # rows that see none of it: equal (an all-or-nothing mask; the maximum they start from is the same)
            assert torch.equal(got[torch.from_numpy(~sees)], clean[torch.from_numpy(~sees)])
    q = rows(rng, 2, H * g, D, torch.bfloat16, dev)
    cache, codes, scales = make_cache(rng, dev, 8, H, page, D)
    clean = w4.kv8_attention(q, cache, t, ints([L], dev))
    q[1, 0, 5] = float("nan")
    got = w4.kv8_attention(q, cache, t, ints([L], dev))
    assert torch.isnan(got[1, 0]).all() and torch.equal(got[0], clean[0]) and torch.equal(got[1, 1], clean[1, 1])


def test_attention_follows_lengths_in_a_graph(dev):
    """Decode steps replayed: append, then attend; lengths, tables and inputs change between replays; two graphs side by side."""
    rng = np.random.default_rng(8)
    B, H, g, D, page = 3, 2, 4, 128, 16
    pages = 64
    freqs = w4.rope_freqs(D, device=dev)
    runs = []
    for _ in range(2):
        cache, codes, scales = make_cache(rng, dev, pages, H, page, D)
        table, t = make_table(rng, dev, pages, [300] * B, page)
        x = rows(rng, B, H * g + 2 * H, D, torch.bfloat16, dev)
        lens, q_out = ints([200, 1, 77], dev), torch.empty(B, H * g, D, dtype=torch.bfloat16, device=dev)
        step = lambda x=x, c=cache, t=t, lens=lens, o=q_out: w4.kv8_attention(  # noqa: E731
            w4.kv8_append(c, x[:, H * g:H * g + H], x[:, H * g + H:], t, lens, q=x[:, :H * g], q_out=o, freqs=freqs), c, t, lens)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((cache, x, lens, graph, out, step))
    streams = [torch.cuda.Stream() for _ in runs]
    for i in range(6):
        for cache, x, lens, *_ in runs:
            lens += 1
            x.copy_(rows(rng, B, H * g + 2 * H, D, torch.bfloat16, dev))
        torch.cuda.synchronize()
        for (_, _, _, graph, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for cache, x, lens, graph, out, step in runs:
            assert torch.equal(out, step())  # appending the same tokens again changes nothing
    w4.w4a4_check()


def test_attention_on_another_stream(dev):
    rng = np.random.default_rng(10)
    lens, counts, page, H, g, D = [3000, 900], [1, 1], 64, 2, 5, 128
    cache, codes, scales = make_cache(rng, dev, 80, H, page, D)
    table, t = make_table(rng, dev, 80, lens, page)
    q = rows(rng, 2, H * g, D, torch.bfloat16, dev)
    want = w4.kv8_attention(q, cache, t, ints(lens, dev))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = w4.kv8_attention(q, cache, t, ints(lens, dev), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    k, v = w4.kv8_read(cache, t, ints(lens, dev), 2, stream=side)
    side.synchronize()
    ref = np.stack([values(codes, scales, table[b], L)[:, -1] for b, L in enumerate(lens)], axis=1)
    assert np.array_equal(k.double().cpu().numpy(), ref[0]) and np.array_equal(v.double().cpu().numpy(), ref[1])


def test_the_largest_batch_and_the_emptiest_table(dev):
    rng = np.random.default_rng(15)
    B, D, page = 2048, 64, 16
    cache, codes, scales = make_cache(rng, dev, 32, 1, page, D)
    lens = [int(x) for x in rng.integers(0, 64, B)]
    table = rng.integers(0, 32, (B, 4)).astype(np.int32)
    q = rows(rng, B, 3, D, torch.bfloat16, dev)
    t = torch.from_numpy(table).to(dev)
    check_attention(w4.kv8_attention(q, cache, t, ints(lens, dev)), q, codes, scales, table, lens, [1] * B)
    many = rows(rng, 2 * B, 9, D, torch.bfloat16, dev)
    check_attention(w4.kv8_attention(many, cache, t, ints(lens, dev)), many, codes, scales, table, lens, [2] * B)
    none = torch.empty(2, 0, dtype=torch.int32, device=dev)
    for n in (1, 30):
        assert (w4.kv8_attention(q[:2 * n], cache, none, ints([0, 0], dev)) == 0).all()
    w4.w4a4_check()


def test_attention_with_a_scale_of_zero_averages(dev):
    rng = np.random.default_rng(16)
    cache, codes, scales = make_cache(rng, dev, 8, 1, 32, 128)
    for n, width in ((2, None), (60, None), (60, WIDE // 32)):
        table, t = make_table(rng, dev, 8, [200], 32, width)
        q = rows(rng, n, 4, 128, torch.bfloat16, dev)
        got = w4.kv8_attention(q, cache, t, ints([200], dev), scale=0.0, dtype=torch.float32)
        check_attention(got, q, codes, scales, table, [200], [n], scale=0.0)


def test_the_first_calls_of_a_process_can_be_captured():
    code = """
import sys; sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch, hadamard_rotated_w4a4_gb300 as w4
cache = w4.alloc_kv8(8, 2, 128, 64)
x = torch.randn(40, 8, 128, device='cuda').bfloat16()
t, lens = torch.arange(4, device='cuda', dtype=torch.int32)[None], torch.tensor([200], device='cuda', dtype=torch.int32)
f = w4.rope_freqs(128)
out = torch.empty(40, 4, 128, device='cuda', dtype=torch.bfloat16)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q = torch.empty_like(out)
    w4.kv8_append(cache, x[:, 4:6], x[:, 6:], t, lens, q=x[:, :4], q_out=q, freqs=f)
    w4.kv8_attention(q, cache, t, lens, out=out)
    one = w4.kv8_attention(q[:1], cache, t, lens)
g.replay(); torch.cuda.synchronize()
a = out.clone()
w4.kv8_attention(q, cache, t, lens, out=out); torch.cuda.synchronize()
assert torch.equal(a, out) and torch.isfinite(out).all() and torch.equal(one, w4.kv8_attention(q[:1], cache, t, lens))
w4.w4a4_check()
print('captured')
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_a_batch_of_many_lengths(dev):
    """More sequences than a scan's width, empty and full ones among them; sharing pages that are only read."""
    rng = np.random.default_rng(11)
    B, H, g, D, page = 700, 1, 2, 64, 16
    cache, codes, scales = make_cache(rng, dev, 64, H, page, D)
    lens = [int(x) for x in rng.integers(0, 128, B)]
    table = rng.integers(0, 64, (B, 8)).astype(np.int32)
    q = rows(rng, B, H * g, D, torch.bfloat16, dev)
    got = w4.kv8_attention(q, cache, torch.from_numpy(table).to(dev), ints(lens, dev))
    check_attention(got, q, codes, scales, table, lens, [1] * B)


def test_offsets_past_32_bits(dev):
    """A cache of more than 2^32 codes, used at its far end."""
    D, page, H = 256, 128, 8
    pages = (1 << 32) // (H * 2 * page * D) + 9
    rng = np.random.default_rng(12)
    codes = torch.empty(pages, H, 2, page, D, dtype=torch.int8, device=dev)
    scales = torch.full((pages, H, 2, page // 16), 121, dtype=torch.uint8, device=dev)
    codes[-8:] = torch.randint(-127, 128, (8, H, 2, page, D), device=dev, dtype=torch.int8)
    cache = w4.KvCache8(codes, scales)
    table = np.arange(pages - 8, pages, dtype=np.int32)[::-1][None].copy()
    lens, counts = [900], [3]
    q = rows(rng, 3, H, D, torch.bfloat16, dev)
    t = torch.from_numpy(table).to(dev)
    tail, ts = codes[-8:].cpu().numpy(), scales[-8:].cpu().numpy()
    got = w4.kv8_attention(q, cache, t, ints(lens, dev))
    check_attention(got, q, tail, ts, table - (pages - 8), lens, counts)
    x = rows(rng, 3, 2 * H, D, torch.bfloat16, dev)
    w4.kv8_append(cache, x[:, :H], x[:, H:], t, ints(lens, dev))
    f = oracle.rotate_h32(x.float().cpu().numpy())
    oracle.kv8_append(tail, ts, f[:, :H], f[:, H:], table - (pages - 8), lens, counts)
    assert np.array_equal(codes[-8:].cpu().numpy(), tail) and np.array_equal(scales[-8:].cpu().numpy(), ts)
