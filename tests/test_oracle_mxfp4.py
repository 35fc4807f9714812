"""The MXFP4 oracle against hand-worked values, brute force and exact fractions (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

import oracle


def test_e2m1_grid_and_every_tie():
    assert oracle.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    # each midpoint goes to its even neighbour, the values next to it to the nearer one
    for mid, even in [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]:
        lo = int(np.searchsorted(oracle.E2M1, mid)) - 1
        got = oracle.e2m1_code(np.array([mid, np.nextafter(mid, 0), np.nextafter(mid, 9), -mid]))
        assert got.tolist() == [even, lo, lo + 1, even + 8]
    assert oracle.e2m1_code(np.array([6.0, 6.01, 7.99, 1e30, -9.0, 0.0, -0.0])).tolist() == [7, 7, 7, 7, 15, 0, 8]


def test_e2m1_is_the_nearest_value():
    v = np.random.default_rng(0).uniform(-6, 6, 4000)
    got = oracle.e2m1_code(v)
    val = np.where(got >= 8, -1, 1) * oracle.E2M1[got & 7]
    grid = np.concatenate([oracle.E2M1, -oracle.E2M1])
    assert np.array_equal(np.abs(val - v), np.abs(v[:, None] - grid).min(axis=1))


def block(*head):
    x = np.zeros((1, 32), np.float32)
    x[0, : len(head)] = head
    return x


def test_quantiser_by_hand():
    # a = 4: E = 0; 5 saturates nothing (ties to 4), 6.5 is past 6, -0.75 ties to the even 1.0
    r = oracle.quantize_mxfp4(block(7.9, 5.0, 6.5, -0.75, 0.3), rotate=False)
    assert r["scales"][0, 0] == 127 and r["q"][0, :6].tolist() == [7, 6, 7, 10, 1, 0]
    assert r["codes"][0, :3].tolist() == [7 | 6 << 4, 7 | 10 << 4, 1]
    r = oracle.quantize_mxfp4(block(3.9999998), rotate=False)  # floor(log2) = 1: E = -1
    assert r["scales"][0, 0] == 126 and r["q"][0, 0] == 7
    r = oracle.quantize_mxfp4(block(), rotate=False)
    assert r["scales"][0, 0] == 0 and not r["q"].any()
    r = oracle.quantize_mxfp4(block(np.float32(2.0) ** -140, 2.0 ** -126), rotate=False)  # E clamps at -127
    assert r["scales"][0, 0] == 0 and r["q"][0, :2].tolist() == [0, 4]
    r = oracle.quantize_mxfp4(block(3.4e38), rotate=False)
    assert r["scales"][0, 0] == 125 + 127
    for bad in (np.nan, np.inf, -np.inf):
        r = oracle.quantize_mxfp4(np.concatenate([block(1.0, bad), block(1.0)], axis=1), rotate=False)
        assert r["scales"][0].tolist() == [255, 125] and not r["q"][0, :32].any() and r["q"][0, 32] == 6
        v = oracle.mxfp4_values(r["codes"], r["scales"])
        assert np.isnan(v[0, :32]).all() and v[0, 32] == 1.0


def test_rotation_is_the_int4_formats():
    x = np.random.default_rng(1).standard_normal((3, 96)).astype(np.float32)
    r = oracle.quantize_mxfp4(x)
    u = oracle.quantize_mxfp4(oracle.rotate_h32(x), rotate=False)
    assert np.array_equal(r["codes"], u["codes"]) and np.array_equal(r["scales"], u["scales"])


@pytest.mark.parametrize("seed", range(3))
def test_round_trip_error(seed):
    # error at most half the spacing (scale/4 to scale), or the 2 lost past 6
    x = np.random.default_rng(seed).standard_normal((5, 160)).astype(np.float32)
    r = oracle.quantize_mxfp4(x)
    y = oracle.rotate_h32(x).astype(np.float64)
    s = np.repeat(np.exp2(r["scales"].astype(np.float64) - 127), 32, axis=1)
    v = np.abs(y) / s
    half = np.where(v < 2, 0.25, np.where(v < 4, 0.5, np.where(v <= 6, 1.0, 2.0)))
    assert (v < 8).all() and (np.abs(oracle.mxfp4_values(r["codes"], r["scales"]) - y) <= half * s).all()


def test_matmul_in_fractions():
    rng = np.random.default_rng(4)
    w, a = oracle.quantize_mxfp4(rng.standard_normal((3, 64))), oracle.quantize_mxfp4(rng.standard_normal((2, 64)))
    Y = oracle.mxfp4_matmul(w, a)

    def value(r, row, k):
        q = int(r["q"][row, k])
        mag = [Fraction(0), Fraction(1, 2), 1, Fraction(3, 2), 2, 3, 4, 6][q & 7]
        return (-1 if q & 8 else 1) * mag * Fraction(2) ** (int(r["scales"][row, k // 32]) - 127)

    for m in range(2):
        for n in range(3):
            want = sum(value(a, m, k) * value(w, n, k) for k in range(64))
            assert Fraction(Y[m, n]) == want
