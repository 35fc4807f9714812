"""Appending at the edges: elements that the positions leave alone, tokens before a sequence's start, and what
w4a4_check says of several faults at once."""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from kv8_testutil import ints, make_cache, make_table
from w4a4_testutil import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def flagged():
    with pytest.raises(w4.W4A4Error) as e:
        w4.w4a4_check()
    return e.value.status_name


@pytest.mark.parametrize("dim,nf,interleaved", [(64, 5, True), (64, 8, False), (128, 1, True), (128, 30, True), (256, 127, True), (256, 120, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_elements_past_the_pairs_pass_as_they_are(dev, dim, nf, interleaved, dtype):
    """Infinities, NaN and zeros of either sign there: bit for bit, and nothing of them in the pairs or in one another."""
    gen = torch.Generator(dev).manual_seed(nf)
    T, Hq, at = 21, 3, 40
    x = torch.randn(T, Hq + 2, dim, device=dev, generator=gen)
    odd = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1.0, -1.0], device=dev)
    n = dim - 2 * nf
    pick = torch.randint(0, 14, (T, Hq, n), device=dev, generator=gen)  # half of them as they are
    x[:, :Hq, 2 * nf:] = torch.where(pick < 7, odd[pick.clamp(max=6)], x[:, :Hq, 2 * nf:])
    x = x.to(dtype)
    cache, t, lens = w4.alloc_kv8(8, 1, dim, 16, dev), ints(range(8), dev)[None], ints([at + T], dev)
    freqs = w4.rope_freqs(2 * nf, device=dev)
    call = lambda q, o: w4.kv8_append(cache, x[:, Hq:Hq + 1], x[:, Hq + 1:], t, lens, q=q, q_out=o, freqs=freqs, interleaved=interleaved)  # noqa: E731
    q = x[:, :Hq]
    got = call(q, torch.empty(T, Hq, dim, dtype=dtype, device=dev))
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    assert torch.equal(got[..., 2 * nf:].isnan(), q[..., 2 * nf:].isnan())
    same = ~q[..., 2 * nf:].isnan()
    assert torch.equal(got[..., 2 * nf:].contiguous().view(bits)[same], q[..., 2 * nf:].contiguous().view(bits)[same])
    clean = q.clone()
    clean[..., 2 * nf:] = 1
    want = call(clean, torch.empty(T, Hq, dim, dtype=dtype, device=dev))
    assert torch.isfinite(got[..., :2 * nf]).all() and torch.equal(got[..., :2 * nf], want[..., :2 * nf])
    mine = q.clone()  # in place
    call(mine, None)
    assert torch.equal(mine.isnan(), got.isnan()) and torch.equal(mine.nan_to_num(nan=5), got.nan_to_num(nan=5))
    w4.w4a4_check()


@pytest.mark.parametrize("lens,counts", [([0], [8]), ([5], [8]), ([0, 30], [4, 4]), ([30, 0], [4, 4]), ([0] * 40 + [30], [0] * 39 + [1, 4]),
                                         ([30] + [0] * 40, [4] + [1] + [0] * 39)])
def test_tokens_before_a_sequences_start_are_reported(dev, lens, counts):
    """... also where there is not one token of the sequence; the other sequences' tokens are written."""
    rng = np.random.default_rng(4)
    page, D, T = 16, 64, sum(counts)
    cache, codes, scales = make_cache(rng, dev, 8, 1, page, D)
    table, t = make_table(rng, dev, 8, lens, page)
    x = torch.randn(T, 3, D, device=dev)
    q_out = torch.full((T, 1, D), 7.0, device=dev)
    for cu in ([0, *np.cumsum(counts)], None):
        if cu is None and len(set(counts)) > 1:
            continue
        w4.w4a4_check()
        w4.kv8_append(cache, x[:, 1:2], x[:, 2:], t, ints(lens, dev), cu=None if cu is None else ints(cu, dev), q=x[:, :1], q_out=q_out)
        assert flagged() == "W4A4_ERR_DEVICE_FLAG"
        w4.w4a4_check()
        at = 0
        for L, n in zip(lens, counts):
            skip = max(n - L, 0)
            assert (q_out[at:at + skip] == 7).all() and torch.equal(q_out[at + skip:at + n], x[at + skip:at + n, :1])
            at += n
    # as many new tokens as there are: nothing to report
    n = min(16, max(lens))
    if n:
        b = lens.index(max(lens))
        w4.kv8_append(cache, x[:1, 1:2].expand(n, 1, D).contiguous(), x[:1, 2:].expand(n, 1, D).contiguous(), t[b:b + 1], ints([n], dev))
    w4.w4a4_check()


def test_a_fault_is_reported_behind_a_wait_that_gave_up(dev):
    rng = np.random.default_rng(5)
    cache, codes, scales = make_cache(rng, dev, 8, 1, 64, 128)
    wide = torch.full((1, (1 << 19) // 64), -1, dtype=torch.int32, device=dev)
    wide[0, :7] = ints(range(7), dev)
    q = torch.randn(50, 2, 128, device=dev).to(torch.bfloat16)
    w4.w4a4_debug_set_wait_limit(2_000_000, 20_000_000)
    try:
        w4.kv8_attention(q, cache, wide, ints([400], dev))
        torch.cuda.synchronize()
    finally:
        w4.w4a4_debug_set_wait_limit()
    w4.kv8_read(cache, wide, ints([500], dev), 100)  # its last page is not one
    assert flagged() == "W4A4_ERR_TIMEOUT"
    assert flagged() == "W4A4_ERR_DEVICE_FLAG"
    w4.w4a4_check()
