"""Attention whose offsets cover a part of the token buffer only: the rows that they name are right, the others as they
were, eager and in one captured graph whose offsets and lengths change between its replays."""
import numpy as np
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from kv8_testutil import check_attention, ints, make_cache, make_table
from w4a4_testutil import device

pytestmark = pytest.mark.gpu

HEADS, GROUP, PAGE = 8, 5, 64
LENS = [5000, 300, 4100]
FULL = None  # all of the buffer


@pytest.fixture(scope="module")
def dev():
    return device()


def counts_of(cover, T):
    return [T - 40, 0, 40] if cover is FULL else cover


def lens_of(counts):
    return [max(L, n) for L, n in zip(LENS, counts)]


def check(out, q, codes, scales, table, lens, counts):
    """The first and the last twelve new tokens of each sequence, and the rows behind the last."""
    at = 0
    for b, (L, n) in enumerate(zip(lens, counts)):
        few = min(n, 12)
        for first in {0, n - few}:  # with a causal mask the first few are a shorter sequence's last
            rows = slice(at + first, at + first + few)
            check_attention(out[rows], q[rows], codes, scales, table[b:b + 1], [L - n + first + few], [few])
        at += n
    assert (out[at:] == 7).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T", [512, 4096])
def test_offsets_cover_a_part_of_the_buffer(dev, dim, T):
    rng = np.random.default_rng(dim + T)
    covers = ([0, 0, 0], [1, 0, 0], [0, 0, 100], [60, 0, 40], [13, 300, 2], FULL)
    pages = sum((max(L, T) + PAGE - 1) // PAGE for L in LENS)
    cache, codes, scales = make_cache(rng, dev, pages, HEADS, PAGE, dim)
    table, t = make_table(rng, dev, pages, [max(L, T) for L in LENS], PAGE)
    q = (torch.randn(T, HEADS * GROUP, dim, device=dev, generator=torch.Generator(dev).manual_seed(dim)) * 0.5).to(torch.bfloat16)
    lens, cu, out = ints(LENS, dev), ints([0] * 4, dev), torch.empty(T, HEADS * GROUP, dim, dtype=torch.bfloat16, device=dev)

    def name(cover):
        counts = counts_of(cover, T)
        lens.copy_(ints(lens_of(counts), dev))
        cu.copy_(ints([0, *np.cumsum(counts)], dev))
        out.fill_(7)
        return counts

    for cover in covers:
        counts = name(cover)
        w4.kv8_attention(q, cache, t, lens, cu=cu, out=out)
        check(out, q, codes, scales, table, lens_of(counts), counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.kv8_attention(q, cache, t, lens, cu=cu, out=out)
    for cover in reversed(covers):
        counts = name(cover)
        graph.replay()
        check(out, q, codes, scales, table, lens_of(counts), counts)
        again = out.clone()
        name(cover)
        w4.kv8_attention(q, cache, t, lens, cu=cu, out=out, ws=None)  # never cut
        check(out, q, codes, scales, table, lens_of(counts), counts)
        name(cover)
        w4.kv8_attention(q, cache, t, lens, cu=cu, out=out)
        assert torch.equal(out, again)
    w4.w4a4_check()


def test_offsets_that_the_device_clamps_leave_no_named_row(dev):
    """Offsets past the buffer, and a batch of more sequences than a warp's lanes whose offsets name a few rows."""
    rng = np.random.default_rng(3)
    dim, T = 128, 512
    lens = [5000] + [17] * 39
    cache, codes, scales = make_cache(rng, dev, 200, HEADS, PAGE, dim)
    table, t = make_table(rng, dev, 200, lens, PAGE)
    q = torch.randn(T, HEADS * GROUP, dim, device=dev).to(torch.bfloat16)
    out = torch.full_like(q, 7)
    counts = [100, 0, 3] + [0] * 37
    w4.kv8_attention(q, cache, t, ints(lens, dev), cu=ints([0, *np.cumsum(counts)], dev), out=out)
    check(out, q, codes, scales, table, lens, counts)
    w4.w4a4_check()
    out.fill_(7)
    w4.kv8_attention(q, cache, t[:1], ints([5000], dev), cu=ints([450, 600], dev), out=out)  # rows 450 .. 511
    with pytest.raises(w4.W4A4Error) as e:
        w4.w4a4_check()
    assert e.value.status_name == "W4A4_ERR_DEVICE_FLAG"
    assert (out[:450] == 7).all()
    check_attention(out[450:], q[450:], codes, scales, table[:1], [5000], [62])
