"""Appending at the edges: elements that the positions leave alone."""
import pytest
import torch

import hadamard_rotated_w4a4_gb300 as w4
from kv8_testutil import ints
from w4a4_testutil import device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


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
