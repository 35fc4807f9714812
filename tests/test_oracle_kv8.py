"""The 8-bit key/value oracle pinned to things other than itself."""
import numpy as np
import pytest

import oracle


def empty(pages=3, heads=2, page=16, dim=64):
    return np.zeros((pages, heads, 2, page, dim), np.int8), np.zeros((pages, heads, 2, page // 16), np.uint8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_of_the_plane(interleaved):
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((5, 2, 64)), 10000.0 ** (-np.arange(0, 64, 2) / 64)
    pos = np.array([0, 1, 7, 100, 65536])
    y = oracle.rope(x, pos, f, interleaved)
    pair = (lambda z: z[..., 0::2] + 1j * z[..., 1::2]) if interleaved else (lambda z: z[..., :32] + 1j * z[..., 32:])
    np.testing.assert_allclose(pair(y), pair(x) * np.exp(1j * pos[:, None] * f)[:, None], atol=1e-9)
    assert np.array_equal(y[0], x[0])


def test_rope_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k, f = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64)), 1e4 ** (-np.arange(0, 64, 2) / 64)
    dots = [(oracle.rope(q, np.array([p + 5]), f, False) * oracle.rope(k, np.array([p]), f, False)).sum() for p in (0, 3, 999)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)


def test_rope_of_fewer_pairs_leaves_the_rest():
    x = np.random.default_rng(2).standard_normal((3, 1, 64))
    y = oracle.rope(x, np.arange(3), np.ones(8), False)
    assert np.array_equal(y[..., 16:], x[..., 16:]) and not np.array_equal(y[1:, :, :16], x[1:, :, :16])


def test_exponent_by_hand():
    for a, e in ((0.0, -40), (127.0, 0), (127.0001, 1), (63.5, -1), (63.6, 0), (1.0, -6), (0.9921875, -7), (1e30, 40), (1e-30, -40)):
        assert oracle.kv8_exponent(a) == e


def test_append_round_trip_and_layout():
    rng = np.random.default_rng(3)
    codes, scales = empty(pages=4, page=32)
    k, v = rng.standard_normal((2, 40, 2, 64))
    table = np.array([[2, 0]])
    oracle.kv8_append(codes, scales, k, v, table, [40], [40])
    back = oracle.kv8_values(codes, scales, table[0], 40)
    for x, y in ((k, back[0]), (v, back[1])):
        for p in range(0, 40, 16):
            amax = np.abs(x[p:p + 16]).max(axis=(0, 2))  # per head
            step = np.exp2(np.ceil(np.log2(amax / 127)))
            assert (np.abs(x[p:p + 16] - y[p:p + 16]) <= step[:, None] / 2).all()
    assert not codes[1].any() and not codes[3].any() and not codes[0, :, :, 8:].any()


def test_growing_scales_stay_within_a_step():
    rng = np.random.default_rng(4)
    codes, scales = empty()
    x = rng.standard_normal((16, 2, 64)) * np.exp2(np.arange(16))[:, None, None]  # each token needs a larger scale
    for t in range(16):
        oracle.kv8_append(codes, scales, x[t:t + 1], -x[t:t + 1], np.array([[1]]), [t + 1], [1])
    back = oracle.kv8_values(codes, scales, [1], 16)
    step = 2.0 ** (scales[1, :, 0, 0].astype(float) - 127)
    assert (np.abs(back[0] - x) < step[:, None]).all() and np.array_equal(back[1], -back[0])


def test_non_finite_rows_poison_their_block_until_it_restarts():
    codes, scales = empty()
    x = np.ones((1, 2, 64))
    bad = x.copy()
    bad[0, 1, 5] = np.inf
    table = np.array([[0]])
    oracle.kv8_append(codes, scales, x, x, table, [1], [1])
    oracle.kv8_append(codes, scales, bad, x, table, [2], [1])
    oracle.kv8_append(codes, scales, x, x, table, [3], [1])
    back = oracle.kv8_values(codes, scales, [0], 3)
    assert np.isnan(back[0][:, 1]).all() and np.isfinite(back[0][:, 0]).all() and np.isfinite(back[1]).all()
    oracle.kv8_append(codes, scales, x, x, table, [1], [1])
    assert np.array_equal(oracle.kv8_values(codes, scales, [0], 1)[0], x)


def test_attention_by_hand():
    rng = np.random.default_rng(5)
    v = rng.standard_normal((6, 1, 8))
    q = rng.standard_normal((2, 3, 8))
    same = np.ones((6, 1, 8))
    out = oracle.kv8_attention(q, same, v, 0.3, True, 0)
    np.testing.assert_allclose(out[1, 2], v[:, 0].mean(axis=0))
    np.testing.assert_allclose(out[0, 0], v[:5, 0].mean(axis=0))
    np.testing.assert_allclose(oracle.kv8_attention(q, same, v, 0.3, False, 0)[0, 0], v[:, 0].mean(axis=0))
    np.testing.assert_allclose(oracle.kv8_attention(q, same, v, 0.3, True, 2)[0, 1], v[3:5, 0].mean(axis=0))
    k = np.zeros((6, 1, 8))
    k[2] = 100.0
    np.testing.assert_allclose(oracle.kv8_attention(np.ones((1, 1, 8)), k, v, 1.0, True, 0)[0, 0], v[2, 0])
    assert not oracle.kv8_attention(q, np.zeros((0, 1, 8)), np.zeros((0, 1, 8)), 1.0, False, 0).any()
    assert not oracle.kv8_attention(np.ones((3, 1, 8)), same[:1], v[:1], 1.0, True, 0)[:2].any()  # before the start
