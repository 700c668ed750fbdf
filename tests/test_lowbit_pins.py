"""The oracle of the 8-bit moments and the 4-bit matrices against worked values (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import lowbit as L


def test_hash_flips_half_of_its_bits():
    i = np.arange(1 << 14, dtype=np.uint64)
    h = L.hash_bits(L.hash_key(7, 3, 1), i)
    for b in (0, 5, 13, 31, 33):
        d = h ^ L.hash_bits(L.hash_key(7, 3, 1), i ^ np.uint64(1 << b))
        share = [((d >> np.uint32(o)) & np.uint32(1)).mean() for o in range(32)]
        # 2^14 draws: five standard deviations are 5 / (2 * 2^7) = 0.02
        assert max(abs(s - 0.5) for s in share) < 0.02, b
    for other in (L.hash_key(8, 3, 1), L.hash_key(7, 4, 1), L.hash_key(7, 3, 2), L.hash_key(7 + (1 << 32), 3, 1)):
        assert abs(np.corrcoef(h.astype(float), L.hash_bits(other, i).astype(float))[0, 1]) < 5 / 128


@pytest.mark.parametrize("second", [False, True])
def test_every_code_survives_a_round_trip(second):
    values = L.code_values(second)
    assert np.all(np.diff(values) > 0) and values[-1] == 1.875 and values[0] == 0
    for e in (-100, 0, 3, 120):
        v = np.zeros(256 if second else 128)
        v[:] = values * 2.0 ** e
        v = v if second else np.concatenate([v, -v])
        groups = v.reshape(-1, 4)                               # 64 groups of 4, each beside the largest code
        w = np.zeros((len(groups), 64))
        w[:, :4], w[:, 4] = groups, 1.875 * 2.0 ** e
        for u in (None, np.zeros(w.size), np.full(w.size, 0.999)):
            c, x = L.encode8(w, second, u)
            assert np.all(x == 127 + e) and np.array_equal(L.decode8(c, x, second), w.reshape(-1))


def test_moment_codes_by_hand():
    v = np.zeros(64)
    v[:6] = [1.9, 1.0, 1.06, 1.07, 2.0 ** -17, 2.0 ** -19]      # past 1.875 it could round up: exponent 1
    c, e = L.encode8(v, False)
    assert e[0] == 128
    got = L.decode8(c, e, False)[:6]
    assert np.array_equal(got, [1.875, 1.0, 1.0, 1.125, 0.0, 0.0])            # the lowest codes are 2^-16 apart, 2^-17 is a tie: to even
    c, e = L.encode8(np.abs(v), True)
    assert np.array_equal(L.decode8(c, e, True)[4:6], [2.0 ** -17, 2.0 ** -19])
    tiny = np.zeros(64)
    tiny[:2] = [1.0, 2.0 ** -40]
    c, e = L.encode8(tiny, True)
    assert c[1] == 1 and L.decode8(c, e, True)[1] == 2.0 ** -33               # never to zero


def test_matrix_elements_by_hand():
    x = np.zeros((2, 40))
    x[0, :10] = [6.9, -6.0, 5.0, 4.9, 3.5, 2.5, 1.25, 0.75, 0.25, -0.3]
    x[1, :3] = [7.0, 6.9, -5.0]
    x[1, 32] = np.inf
    v, s = L.mx_quantize(x)
    assert s.tolist() == [[127, 1], [128, 255]]
    assert np.array_equal(v[0, :10], [6, -6, 4, 4, 4, 2, 1, 1, 0, -0.5])
    assert np.array_equal(v[1, :3], [8, 6, -4]) and np.isnan(v[1, 32:]).all()     # 3.5 and 2.5 are ties
    v, s = L.mx_quantize(x[:1], np.zeros((1, 40)))
    assert s[0, 0] == 128 and v[0, 0] == 6 and v[0, 2] == 4
    v, _ = L.mx_quantize(x[:1], np.full((1, 40), 0.9999))
    assert v[0, 0] == 8 and v[0, 1] == -6 and v[0, 8] == 1


def test_stochastic_rounding_keeps_the_expectation():
    rng = np.random.default_rng(1)
    n = 1 << 16
    x = np.tile(np.concatenate([[5.9], rng.uniform(0, 6, 31)]), (n // 32, 1))
    u = (L.hash_bits(L.hash_key(3, 0, 0), np.arange(n)) >> 10).reshape(-1, 32) * 2.0 ** -22
    v, _ = L.mx_quantize(x, u)
    # steps of at most 2: standard deviation at most 1 of an element, 2048 of each
    assert np.abs(v.mean(0) - x[0]).max() < 5 / np.sqrt(n // 32)
    c, e = L.encode8(np.concatenate([x.reshape(-1)]), True, u.reshape(-1))
    got = L.decode8(c, e, True).reshape(-1, 32).mean(0)
    assert np.abs(got - x[0]).max() < 5 * 0.25 / np.sqrt(n // 32)             # steps of at most 0.5
    for kind, bits in (("bf16", 7), ("f16", 10)):
        y = np.full(n, 1.0 + 0.3 * 2.0 ** -bits)
        w = L.round16(y, kind, u.reshape(-1))
        assert set(np.unique(w)) == {1.0, 1.0 + 2.0 ** -bits}
        assert abs(w.mean() - y[0]) < 5 * 0.5 * 2.0 ** -bits / np.sqrt(n)


def test_a_lost_group_reads_as_nan_and_is_taken_up_as_the_largest_value():
    c = np.full(192, 77, np.uint8)
    e1, e2 = np.array([130, 140, 255], np.uint8), np.array([131, 255, 140], np.uint8)
    assert np.isnan(L.decode8(c, e1, False)[128:]).all() and np.isnan(L.decode8(c, e2, True)[64:128]).all()
    m1, m2 = L.carried8(c, e1, c, e2)
    assert np.array_equal(m1[:64], L.decode8(c, e1, False)[:64]) and (m1[64:] == 0).all()
    assert np.array_equal(m2[:64], L.decode8(c, e2, True)[:64]) and (m2[64:128] == 1.875 * 2.0 ** 127).all()
    assert np.array_equal(m2[128:], L.decode8(c, e2, True)[128:])
